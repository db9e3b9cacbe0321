"""Newton-Schulz orthogonalisation and the Muon step against a plain fp64
implementation, on cuda:0.

Tolerances (relative, Frobenius norm per matrix).

fp32 weights.  Every factor is held to 22 bits, so each step adds an error of
at most about 4 roundings (X, A, B and the product's sum) of 2^-22 of its X's
norm, and each later step multiplies it by at most its largest slope, a =
3.4445.  ||X_k||_F is at most a^k (as ||X_0||_F = 1) and at most 1.21 sqrt(m)
(no singular value passes 1.21), so
  error <= 4 2^-22 sum_k a^(n-k) min(a^k, 1.21 sqrt(m)).

bf16 weights.  Rounding the result to bf16 is off by at most half a step, 2^-8;
A and B as one fp16 (half a step 2^-11 each) act on the last two steps' X
without amplification: 4 2^-11 more.
"""
import math

import numpy as np
import pytest
import torch

from gradient_all_reduce_ar_amd import _binding as B

DEV = "cuda:0"
T = {"fp32": torch.float32, "bf16": torch.bfloat16}
COEF = (3.4445, -4.7750, 2.0315)


def orthogonalized(u, steps):
    """The definition, fp64."""
    x = u.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t().contiguous() if tall else x
    x = x / (x.norm() + 1e-7)
    for a, b, c in steps:
        g = x @ x.t().contiguous()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.t().contiguous() if tall else x


def tolerance(want, weight, n=5):
    if weight == "bf16":
        return 2.0 ** -8 + 4 * 2.0 ** -11
    a, m = COEF[0], min(want.shape)
    grown = sum(a ** (n - k) * min(a ** k, 1.21 * math.sqrt(m)) for k in range(n + 1))
    return 4 * 2.0 ** -22 * grown / max(float(want.norm()), 1e-3)


def matrices(shapes, kind, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    out = []
    for r, c in shapes:
        m = torch.randn((r, c), generator=g, device=DEV)
        if kind == "low_rank":
            k = max(1, min(r, c) // 16)
            m = torch.randn((r, k), generator=g, device=DEV) @ torch.randn((k, c), generator=g, device=DEV) + 0.05 * m
        elif kind == "tiny":
            m = m * 1e-20
        elif kind == "huge":
            m = m * 1e30
        elif kind == "sparse":
            m = m * (torch.rand((r, c), generator=g, device=DEV) < 0.05)
        out.append(m)
    return out


def arena(mats, offsets, count, dtype, fill=0.0):
    flat = torch.full((count,), fill, device=DEV, dtype=T[dtype])
    for m, at in zip(mats, offsets):
        flat[at:at + m.numel()] = m.reshape(-1).to(T[dtype])
    return flat


def back_to_back(shapes):
    offs = np.concatenate([[0], np.cumsum([r * c for r, c in shapes])])
    return [int(o) for o in offs[:-1]], int(offs[-1])


def check(got, want, tol, what):
    off = float((got.double() - want).norm()) / max(float(want.norm()), 1e-30)
    assert off <= tol, f"{what}: {off:.3g} off, {tol:.3g} allowed"


SHAPES = [
    [(1, 1)], [(1, 7)], [(9, 1)], [(64, 64)], [(33, 47), (47, 33), (1, 5), (64, 128), (128, 64)], [(65, 129)],
    [(130, 66)], [(255, 515)], [(300, 200), (16, 16), (200, 300)], [(8, 2048)], [(2048, 8)], [(512, 768), (768, 512)],
    [(64, 64)] * 20, [(1024, 1024)], [(128, 128), (1, 300)], [(64, 512), (512, 60)], [(65, 500)], [(96, 256)] * 3,
    [(1, 1), (33, 47), (600, 300), (5, 3), (64, 64), (1, 700), (700, 1)],  # small ones beside one that is not
]


@pytest.mark.gpu
@pytest.mark.parametrize("grad,weight", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "bf16")])
@pytest.mark.parametrize("shapes", SHAPES, ids=lambda s: "+".join(f"{r}x{c}" for r, c in s[:3]) + f"-{len(s)}")
def test_orthogonalize(shapes, grad, weight):
    print("case", shapes, grad, weight, flush=True)
    offs, n = back_to_back(shapes)
    g = arena(matrices(shapes, "normal"), offs, n, grad)
    out = torch.full((n,), 7.0, device=DEV, dtype=T[weight])
    plan = B.ar_muon_plan_create(shapes, grad, weight)
    B.ar_orthogonalize(plan, g, out)
    torch.cuda.synchronize()
    for (r, c), at in zip(shapes, offs):
        want = orthogonalized(g[at:at + r * c].view(r, c), [COEF] * 5)
        check(out[at:at + r * c].view(r, c), want, tolerance(want, weight), f"{r}x{c}")
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("weight", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["low_rank", "tiny", "huge", "sparse"])
def test_spectra_and_sizes(kind, weight):
    """Few large singular values, gradients far below and above 1, mostly zeros.  1e-20 lies below the norm's
    1e-7, which then sets the scale."""
    shapes = [(128, 192), (192, 128), (65, 64)]
    offs, n = back_to_back(shapes)
    g = arena(matrices(shapes, kind), offs, n, "fp32")
    out = torch.empty(n, device=DEV, dtype=T[weight])
    plan = B.ar_muon_plan_create(shapes, "fp32", weight)
    B.ar_orthogonalize(plan, g, out)
    torch.cuda.synchronize()
    for (r, c), at in zip(shapes, offs):
        want, got = orthogonalized(g[at:at + r * c].view(r, c), [COEF] * 5), out[at:at + r * c].view(r, c)
        if kind == "tiny":  # X_0 is 1e-13: hi + lo keep 2^-39 of the bound 1 (2^-14 2^-25), amplified by a^5
            assert float((got.double() - want).abs().max()) <= COEF[0] ** 5 * 2.0 ** -38
        else:
            check(got, want, tolerance(want, weight), f"{kind} {r}x{c}")
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("grad,weight", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16")])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("inplace", [True, False])
def test_step(grad, weight, nesterov, inplace):
    """Momentum, Nesterov, weight decay, grad_scale and the scales; at odd offsets with gaps that stay."""
    shapes = [(96, 160), (160, 96), (33, 65), (5, 3)]
    offs, at = [], 3
    for r, c in shapes:
        offs.append(at)
        at += r * c + 5
    n = at
    lr, mu, decay, gs = 0.05, 0.9, 0.1, 1 / 16
    g = arena(matrices(shapes, "normal", 1), offs, n, grad, 7.0)
    m0 = arena(matrices(shapes, "normal", 2), offs, n, "fp32", 7.0)
    w0 = arena(matrices(shapes, "normal", 3), offs, n, weight, 7.0)
    m, w = m0.clone(), w0.clone()
    mo = m if inplace else torch.full_like(m, 7.0)
    wo = w if inplace else torch.full_like(w, 7.0)
    plan = B.ar_muon_plan_create(shapes, grad, weight, offs)
    B.ar_muon_step(plan, g, m, w, lr, mu=mu, weight_decay=decay, grad_scale=gs, nesterov=nesterov,
                   momentum_out=None if inplace else mo, weights_out=None if inplace else wo)
    torch.cuda.synchronize()
    if not inplace:
        assert torch.equal(m, m0) and torch.equal(w, w0)
    held = torch.zeros(n, dtype=torch.bool, device=DEV)
    for (r, c), at in zip(shapes, offs):
        part = slice(at, at + r * c)
        held[part] = True
        gd, md, wd = g[part].double() * gs, m0[part].double(), w0[part].double()
        m1 = mu * md + gd
        # three fp32 roundings (2^-24 each) of terms no larger than |mu m| + |g|
        assert ((mo[part].double() - m1).abs() <= 4 * 2.0 ** -24 * (mu * md.abs() + gd.abs())).all()
        o = orthogonalized((gd + mu * m1 if nesterov else m1).view(r, c), [COEF] * 5)
        scale = math.sqrt(max(1, r / c))
        want = (1 - lr * decay) * wd.view(r, c) - lr * scale * o
        half = torch.finfo(T[weight]).eps / 2
        tol = lr * scale * tolerance(o, weight) * float(o.norm()) + (half + 4 * 2.0 ** -24) * float(want.norm())
        assert float((wo[part].view(r, c).double() - want).norm()) <= tol
    for t in (mo, wo):
        assert (t[~held].double() == 7).all(), "the gaps changed"
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("steps", [[COEF], [COEF] * 2, [COEF] * 7, [(1.5, -0.5, 0.0)] * 6, [(2.0, -1.5, 0.5)] * 3 + [COEF]])
@pytest.mark.parametrize("weight", ["fp32", "bf16"])
def test_iterations(steps, weight):
    """Other numbers of steps and other coefficients (each with |slope| at most 3.4445 on the way)."""
    shapes = [(70, 100), (64, 32)]
    offs, n = back_to_back(shapes)
    g = arena(matrices(shapes, "normal", 4), offs, n, "fp32")
    out = torch.empty(n, device=DEV, dtype=T[weight])
    plan = B.ar_muon_plan_create(shapes, "fp32", weight)
    B.ar_orthogonalize(plan, g, out)  # with the default steps first: the change takes effect on a used plan
    B.ar_muon_plan_set_iterations(plan, len(steps), steps)
    B.ar_orthogonalize(plan, g, out)
    torch.cuda.synchronize()
    for (r, c), at in zip(shapes, offs):
        want = orthogonalized(g[at:at + r * c].view(r, c), steps)
        check(out[at:at + r * c].view(r, c), want, tolerance(want, weight, len(steps)), f"{r}x{c}")
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
def test_scales():
    shapes = [(64, 64), (0, 9), (32, 96)]
    offs, n = back_to_back(shapes)
    g = arena(matrices(shapes, "normal", 5), offs, n, "fp32")
    plan = B.ar_muon_plan_create(shapes, "fp32", "fp32")
    outs = []
    for scales in (None, [3.0, 9.0, 0.5], None):
        B.ar_muon_plan_set_scales(plan, scales)
        m, w = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
        B.ar_muon_step(plan, g, m, w, 1.0)
        torch.cuda.synchronize()
        outs.append(w)
    B.ar_muon_plan_destroy(plan)
    assert torch.equal(outs[0], outs[2])
    for k, f in ((0, 3.0), (2, 0.5)):
        part = slice(offs[k], offs[k] + shapes[k][0] * shapes[k][1])
        assert ((outs[1][part] - f * outs[0][part]).abs() <= 2.0 ** -22 * outs[1][part].abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("weight", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_bad_values_stay_in_their_matrix(weight, bad):
    shapes = [(64, 96), (70, 50), (64, 96)]
    offs, n = back_to_back(shapes)
    g = arena(matrices(shapes, "normal", 6), offs, n, "fp32")
    plan = B.ar_muon_plan_create(shapes, "fp32", weight)
    clean, out = torch.empty(n, device=DEV, dtype=T[weight]), torch.empty(n, device=DEV, dtype=T[weight])
    B.ar_orthogonalize(plan, g, clean)
    g[offs[1] + 123] = bad
    B.ar_orthogonalize(plan, g, out)
    torch.cuda.synchronize()
    mid = slice(offs[1], offs[2])
    assert out[mid].isnan().all()
    assert torch.equal(out[:offs[1]], clean[:offs[1]]) and torch.equal(out[offs[2]:], clean[offs[2]:])
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("weight", ["fp32", "bf16"])
def test_zero_gradient(weight):
    shapes = [(64, 96), (33, 1)]
    _, n = back_to_back(shapes)
    plan = B.ar_muon_plan_create(shapes, "bf16", weight)
    out = torch.full((n,), 7.0, device=DEV, dtype=T[weight])
    B.ar_orthogonalize(plan, torch.zeros(n, device=DEV, dtype=torch.bfloat16), out)
    torch.cuda.synchronize()
    assert (out == 0).all()
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
def test_nothing_to_do():
    for shapes in ([], [(0, 4), (5, 0)]):
        plan = B.ar_muon_plan_create(shapes, "fp32", "fp32")
        t = torch.empty(0, device=DEV)
        B.ar_orthogonalize(plan, t, t)
        B.ar_muon_step(plan, t, t, t, 0.1)
        B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_in_place(dtype):
    shapes = [(64, 96), (96, 64), (31, 45)]
    offs, n = back_to_back(shapes)
    g = arena(matrices(shapes, "normal", 7), offs, n, dtype)
    plan = B.ar_muon_plan_create(shapes, dtype, dtype)
    out = torch.empty_like(g)
    B.ar_orthogonalize(plan, g, out)
    B.ar_orthogonalize(plan, g, g)
    torch.cuda.synchronize()
    assert torch.equal(g, out)
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("shapes", [[(64, 64)] * 2, [(160, 224), (96, 64)]])
def test_graph_replays(shapes):
    """A captured step on a stream of its own, replayed with new gradients between eager steps of the same plan."""
    _, n = back_to_back(shapes)
    plan = B.ar_muon_plan_create(shapes, "bf16", "fp32")
    B.ar_muon_plan_prepare(plan)
    g, m, w = torch.empty(n, device=DEV, dtype=torch.bfloat16), torch.zeros(n, device=DEV), torch.randn(n, device=DEV)
    m2, w2 = m.clone(), w.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.ar_muon_step(plan, g, m, w, 0.1, weight_decay=0.1, stream=s)
    for _ in range(4):
        g.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        B.ar_muon_step(plan, g, m2, w2, 0.1, weight_decay=0.1)
        torch.cuda.synchronize()
        assert torch.equal(m, m2) and torch.equal(w, w2)
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("shapes", [[(64, 64), (32, 32)], [(160, 224), (96, 64)]])
def test_captured_step_takes_new_scales(shapes):
    offs, n = back_to_back(shapes)
    plan = B.ar_muon_plan_create(shapes, "fp32", "fp32")
    B.ar_muon_plan_prepare(plan)
    g, m, w = torch.randn(n, device=DEV), torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    m2, w2 = m.clone(), w.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.ar_muon_step(plan, g, m, w, 0.1, stream=s)
    for scales in (None, [0.5, 3.0], [2.0, 0.25], None):
        B.ar_muon_plan_set_scales(plan, scales)
        graph.replay()
        torch.cuda.synchronize()
        B.ar_muon_step(plan, g, m2, w2, 0.1)
        torch.cuda.synchronize()
        assert torch.equal(m, m2) and torch.equal(w, w2)
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("address", [False, True])
def test_capture_needs_a_prepared_plan(address):
    plan = B.ar_muon_plan_create([(96, 64)], "fp32", "fp32")
    g, out, other = torch.randn(96 * 64, device=DEV), torch.zeros(96 * 64, device=DEV), torch.zeros(4, device=DEV)
    args = (g.data_ptr(), out.data_ptr()) if address else (g, out)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        with pytest.raises(B.ArError if address else ValueError):
            B.ar_orthogonalize(plan, *args, stream=s)
        other.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert other.tolist() == [1] * 4 and not out.any() and B.ar_muon_plan_stats(plan)["device"] == -1
    B.ar_orthogonalize(plan, *args)
    torch.cuda.synchronize()
    assert out.any()
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
def test_arena_past_32_bits():
    shapes, at = [(40, 64), (64, 40)], (1 << 32) + 5
    plan = B.ar_muon_plan_create(shapes, "bf16", "bf16", [1, at])
    n = at + 2560
    g = torch.zeros(n, device=DEV, dtype=torch.bfloat16)
    for o in (1, at):
        g[o:o + 2560].normal_()
    out = torch.empty_like(g)
    B.ar_orthogonalize(plan, g, out)
    torch.cuda.synchronize()
    for (r, c), o in zip(shapes, (1, at)):
        want = orthogonalized(g[o:o + 2560].view(r, c), [COEF] * 5)
        check(out[o:o + 2560].view(r, c), want, tolerance(want, "bf16"), f"{r}x{c}")
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
def test_same_bits_every_time():
    shapes = [(200, 300), (300, 200), (64, 64)]
    _, n = back_to_back(shapes)
    g = torch.randn(n, device=DEV)
    outs = []
    for _ in range(3):
        plan = B.ar_muon_plan_create(shapes, "fp32", "fp32")
        outs.append(torch.empty(n, device=DEV))
        B.ar_orthogonalize(plan, g, outs[-1])
        torch.cuda.synchronize()
        B.ar_muon_plan_destroy(plan)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.gpu
def test_experts_reduce_then_step():
    """A training step's path over one arena layout: every rank's expert weight gradients go into its bucketed
    arena, the buckets are all-reduced, Muon updates the experts' weights, and the next forward uses them."""
    ranks, e, inf, outf, tokens = 4, 3, 64, 96, 150
    shapes = [(outf, inf)] * e
    bp = B.ar_bucket_plan_create(ranks, 1, [inf * outf] * e, "fp32", "ring", 2 * inf * outf * 4)
    offs, count = B.ar_bucket_layout(bp, e)
    ex = B.ar_experts_create(e, inf, outf, "fp32", "fp32", offs)
    mu = B.ar_muon_plan_create(shapes, "fp32", "fp32", offs)
    arenas = [torch.zeros(count, device=DEV) for _ in range(ranks)]
    w, m = torch.randn(count, device=DEV), torch.zeros(count, device=DEV)
    w0 = w.clone()
    s = torch.cuda.Stream()
    rng, want, data = np.random.default_rng(3), [torch.zeros(outf, inf, dtype=torch.float64, device=DEV) for _ in range(e)], []
    for r in range(ranks):
        x, dy = torch.randn(tokens, inf, device=DEV), torch.randn(tokens, outf, device=DEV)
        counts = rng.multinomial(tokens, [0.5, 0.2, 0.3])
        data.append((x, dy, torch.from_numpy(np.cumsum(counts).astype(np.int32)).to(DEV)))
        lo = 0
        for k, n in enumerate(counts):
            want[k] += dy[lo:lo + n].double().t().contiguous() @ x[lo:lo + n].double()
            lo += n
    torch.cuda.synchronize()
    ready = [torch.cuda.Event() for _ in range(B.ar_bucket_count(bp))]
    for (x, dy, ends), a in zip(data, arenas):
        B.ar_experts_weight_grad(ex, x, dy, a, ends, stream=s)
    for ev in ready:
        ev.record(s)
    side = torch.cuda.Stream()
    B.ar_bucket_allreduce_after(bp, arenas, side, ready)
    B.ar_muon_step(mu, arenas[ranks - 1], m, w, 0.1, mu=0.0, grad_scale=1 / ranks, nesterov=False, stream=side)
    y = torch.empty(tokens, outf, device=DEV)
    B.ar_experts_forward(ex, data[0][0], w, y, data[0][2], side)
    torch.cuda.synchronize()
    ends = [0] + data[0][2].tolist()
    for k in range(e):
        part = slice(offs[k], offs[k] + inf * outf)
        for a in arenas:
            # sums of `tokens` products per rank and of the ranks, in fp32
            assert float((a[part].view(outf, inf).double() - want[k]).norm()) <= 2.0 ** -18 * float(want[k].norm())
        o = orthogonalized(want[k] / ranks, [COEF] * 5)
        wd = w0[part].view(outf, inf).double() - 0.1 * math.sqrt(outf / inf) * o
        # the gradient's own error (2^-18) is amplified by at most a^5 of ||X_0||_F = 1
        tol = 0.1 * math.sqrt(outf / inf) * (tolerance(o, "fp32") * float(o.norm()) + COEF[0] ** 5 * 2.0 ** -18)
        assert float((w[part].view(outf, inf).double() - wd).norm()) <= tol + 2.0 ** -22 * float(wd.norm())
        rows = slice(ends[k], ends[k + 1])
        ref = data[0][0][rows].double() @ w[part].view(outf, inf).double().t().contiguous()
        assert float((y[rows].double() - ref).norm()) <= 2.0 ** -18 * float(ref.norm())
    B.ar_bucket_plan_destroy(bp)
    B.ar_experts_destroy(ex)
    B.ar_muon_plan_destroy(mu)


@pytest.mark.gpu
@pytest.mark.parametrize("grad", ["fp32", "bf16"])
@pytest.mark.parametrize("shapes", [[(64, 64)] * 4, [(33, 47), (128, 128), (9, 300)], [(300, 200), (160, 224)],
                                    [(1030, 1100)]], ids=lambda s: "+".join(f"{r}x{c}" for r, c in s[:3]))
def test_bf16_results_are_the_fp32_ones_rounded_once(shapes, grad):
    """bf16 weights are computed with the factors that fp32 weights have: the same numbers, rounded once."""
    offs, n = back_to_back(shapes)
    g = arena(matrices(shapes, "normal", 8), offs, n, grad)
    w = arena(matrices(shapes, "normal", 9), offs, n, "bf16")
    res = {}
    for weight in ("fp32", "bf16"):
        plan = B.ar_muon_plan_create(shapes, grad, weight)
        out, m, w1 = torch.empty(n, device=DEV, dtype=T[weight]), torch.ones(n, device=DEV), w.to(T[weight])
        B.ar_orthogonalize(plan, g, out)
        B.ar_muon_step(plan, g, m, w1, 0.1, weight_decay=0.1)
        torch.cuda.synchronize()
        res[weight] = out, m, w1
        B.ar_muon_plan_destroy(plan)
    for wide, narrow, what in zip(res["fp32"], res["bf16"], ("orthogonalised", "momentum", "weights")):
        differ = int((wide.to(narrow.dtype) != narrow).sum())
        assert differ == 0, f"{what}: {differ} of {n} elements differ"


@pytest.mark.gpu
@pytest.mark.parametrize("grad,weight", [("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("steps", [[COEF] * 5, [COEF] * 9, [COEF], [(1.5, -0.5, 0.0)] * 6], ids=["5", "9", "1", "cubic"])
@pytest.mark.parametrize("shapes", [[(64, 40)] * 8, [(64, 64), (33, 47), (60, 130), (128, 128)] * 2, [(128, 192), (192, 128)] * 4],
                         ids=["tiny", "small", "tiled"])
def test_norms_far_below_the_constant(shapes, steps, grad, weight):
    """Matrices of norms from 1 down to 1e-33 in one plan: below 1e-7 that constant divides, X_0 is smaller than 1
    by as much, and the results are still right relative to themselves.  The tolerance is the one above with
    ||X_0||_F = r: ||X_k||_F is at most a^k r."""
    offs, n = back_to_back(shapes)
    norms = [1.0, 1e-7, 1e-9, 1e-11, 1e-13, 1e-17, 1e-25, 1e-33]
    mats = [m * (v / float(m.double().norm())) for m, v in zip(matrices(shapes, "normal", 10), norms)]
    g = arena(mats, offs, n, grad)
    out, m, w = torch.full((n,), 7.0, device=DEV, dtype=T[weight]), torch.zeros(n, device=DEV), torch.zeros(n, device=DEV, dtype=T[weight])
    plan = B.ar_muon_plan_create(shapes, grad, weight)
    B.ar_muon_plan_set_iterations(plan, len(steps), steps)
    assert (B.ar_muon_plan_stats(plan)["launches"] == 1) == (shapes[0] != (128, 192))
    B.ar_orthogonalize(plan, g, out)
    B.ar_muon_plan_set_scales(plan, [1.0] * len(shapes))
    B.ar_muon_step(plan, g, m, w, 0.5, mu=0.0, nesterov=False)
    torch.cuda.synchronize()
    a, top, k = (steps[0][0], 1.21 if steps[0] == COEF else 1.0, len(steps))
    for (r, c), at, norm in zip(shapes, offs, norms):
        u = g[at:at + r * c].view(r, c)
        want, x0 = orthogonalized(u, steps), float(u.double().norm())
        x0 /= x0 + 1e-7
        grown = sum(a ** (k - i) * min(a ** i * x0, top * math.sqrt(min(r, c))) for i in range(k + 1))
        tol = 4 * 2.0 ** -22 * grown / float(want.norm()) + (2.0 ** -8 if weight == "bf16" else 2.0 ** -24)
        assert tol < 0.5
        check(out[at:at + r * c].view(r, c), want, tol, f"{r}x{c} of norm {norm}")
        check(w[at:at + r * c].view(r, c), -0.5 * want, tol, f"step of {r}x{c} of norm {norm}")
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
def test_tensors_of_another_type_are_refused():
    plan = B.ar_muon_plan_create([(8, 16)], "bf16", "fp32")
    g, m, w = (torch.zeros(128, device=DEV, dtype=d) for d in (torch.bfloat16, torch.float32, torch.float32))
    for bad in (dict(g=g.half()), dict(g=g.view(torch.int16)), dict(m=m.int()), dict(w=w.int()), dict(w=w.double())):
        a = dict(g=g, m=m, w=w) | bad
        with pytest.raises(ValueError, match="bfloat16|float32"):
            B.ar_muon_step(plan, a["g"], a["m"], a["w"], 0.1)
    B.ar_muon_plan_destroy(plan)
