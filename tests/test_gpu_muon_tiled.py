"""The tiled Newton-Schulz and Muon kernels (plans of more than one launch)
against fp64, on cuda:0: every tile shape, whole and cut, with edges, wide,
tall and mixed.  Which kernels a list of matrices runs is checked against the
plan, so that a change of the choice shows here.  Tolerances as in
test_gpu_muon.py."""
import math

import numpy as np
import pytest
import torch

from gradient_all_reduce_ar_amd import _binding as B
from tests.test_gpu_muon import COEF, DEV, T, arena, back_to_back, check, matrices, orthogonalized, tolerance
from tests.test_operators_cpu import TILED


def planned(name, grad, weight, offsets=None):
    """A plan of the named matrices, which runs the tiles that it is named for."""
    shapes, want = TILED[name]
    plan = B.ar_muon_plan_create(shapes, grad, weight, offsets)
    for product, (tile, split) in enumerate(want):
        w = B.ar_muon_plan_work(plan, product)
        assert (w["tile"], bool((w["slot"] >= 0).any())) == (tile, split)
    return plan


def gapped(shapes, first=3, gap=5):
    """Odd offsets with gaps, and the arena's size."""
    offs, at = [], first
    for r, c in shapes:
        offs.append(at)
        at += r * c + gap
    return offs, at


@pytest.mark.gpu
@pytest.mark.parametrize("grad,weight", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16")])
@pytest.mark.parametrize("kind", ["normal", "low_rank"])
@pytest.mark.parametrize("name", TILED)
def test_orthogonalize(name, kind, grad, weight):
    print("case", name, kind, grad, weight, flush=True)
    shapes = TILED[name][0]
    offs, n = back_to_back(shapes)
    g = arena(matrices(shapes, kind, 1), offs, n, grad)
    out = torch.full((n,), 7.0, device=DEV, dtype=T[weight])
    plan = planned(name, grad, weight)
    B.ar_orthogonalize(plan, g, out)
    torch.cuda.synchronize()
    for (r, c), at in zip(shapes, offs):
        want = orthogonalized(g[at:at + r * c].view(r, c), [COEF] * 5)
        check(out[at:at + r * c].view(r, c), want, tolerance(want, weight), f"{r}x{c}")
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("grad,weight", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16")])
@pytest.mark.parametrize("nesterov,inplace", [(True, False), (False, True)])
@pytest.mark.parametrize("name", TILED)
def test_step(name, grad, weight, nesterov, inplace):
    """Momentum, Nesterov, weight decay, grad_scale and the scales; at odd offsets with gaps that stay."""
    print("case", name, grad, weight, nesterov, inplace, flush=True)
    shapes = TILED[name][0]
    offs, n = gapped(shapes)
    lr, mu, decay, gs = 0.05, 0.9, 0.1, 1 / 16
    g = arena(matrices(shapes, "normal", 2), offs, n, grad, 7.0)
    m0 = arena(matrices(shapes, "normal", 3), offs, n, "fp32", 7.0)
    w0 = arena(matrices(shapes, "normal", 4), offs, n, weight, 7.0)
    w0.mul_(2.0 ** -6)
    m, w = m0.clone(), w0.clone()
    mo = m if inplace else torch.full_like(m, 7.0)
    wo = w if inplace else w0.clone()
    plan = planned(name, grad, weight, offs)
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
        tol = lr * scale * tolerance(o, "fp32") * float(o.norm()) + (half + 4 * 2.0 ** -24) * float(want.norm())
        assert float((wo[part].view(r, c).double() - want).norm()) <= tol, f"{r}x{c}"
    assert torch.equal(mo[~held], m0[~held]) and torch.equal(wo[~held], w0[~held]), "the gaps changed"
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("steps", [[COEF], [COEF] * 7, [(1.5, -0.5, 0.0)] * 6, [(2.0, -1.5, 0.5)] * 3 + [COEF]])
@pytest.mark.parametrize("name,weight", [("small", "fp32"), ("small", "bf16"), ("square", "fp32"), ("long", "bf16")])
def test_iterations(name, weight, steps):
    """Other numbers of steps and other coefficients, on a plan that has run with the default ones."""
    shapes = TILED[name][0]
    offs, n = back_to_back(shapes)
    g = arena(matrices(shapes, "normal", 5), offs, n, "fp32")
    out = torch.empty(n, device=DEV, dtype=T[weight])
    plan = planned(name, "fp32", weight)
    B.ar_orthogonalize(plan, g, out)
    B.ar_muon_plan_set_iterations(plan, len(steps), steps)
    B.ar_orthogonalize(plan, g, out)
    torch.cuda.synchronize()
    for (r, c), at in zip(shapes, offs):
        want = orthogonalized(g[at:at + r * c].view(r, c), steps)
        check(out[at:at + r * c].view(r, c), want, tolerance(want, weight, len(steps)), f"{r}x{c}")
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["small", "mixed", "large"])
def test_scales(name):
    shapes = TILED[name][0]
    offs, n = back_to_back(shapes)
    g = arena(matrices(shapes, "normal", 6), offs, n, "fp32")
    plan = planned(name, "fp32", "fp32")
    new = [3.0, 0.5, 7.0, 0.25, 2.0][:len(shapes)]
    outs = []
    for scales in (None, new, None):
        B.ar_muon_plan_set_scales(plan, scales)
        m, w = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
        B.ar_muon_step(plan, g, m, w, 1.0)
        torch.cuda.synchronize()
        outs.append(w)
    B.ar_muon_plan_destroy(plan)
    assert torch.equal(outs[0], outs[2])
    for (r, c), at, f in zip(shapes, offs, new):
        part, was = slice(at, at + r * c), math.sqrt(max(1, r / c))
        # w = -scale o, both scales and both results rounded to fp32
        assert ((outs[1][part] * was - f * outs[0][part]).abs() <= 2.0 ** -21 * (f * outs[0][part]).abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("weight", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("name", ["small", "mixed", "large"])
def test_bad_values_stay_in_their_matrix(name, weight, bad):
    shapes = TILED[name][0]
    offs, n = back_to_back(shapes)
    g = arena(matrices(shapes, "normal", 7), offs, n, "fp32")
    plan = planned(name, "fp32", weight)
    clean, out = torch.empty(n, device=DEV, dtype=T[weight]), torch.empty(n, device=DEV, dtype=T[weight])
    B.ar_orthogonalize(plan, g, clean)
    g[offs[1] + 123] = bad
    B.ar_orthogonalize(plan, g, out)
    torch.cuda.synchronize()
    mid = slice(offs[1], offs[2])
    assert out[mid].isnan().all()
    assert torch.equal(out[:offs[1]], clean[:offs[1]]) and torch.equal(out[offs[2]:], clean[offs[2]:])
    # and a used workspace holds nothing of it for the next call
    g[offs[1] + 123] = 0.5
    B.ar_orthogonalize(plan, g, out)
    torch.cuda.synchronize()
    assert out.isfinite().all()
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("weight", ["fp32", "bf16"])
@pytest.mark.parametrize("name", ["small", "long"])
def test_zero_gradient(name, weight):
    _, n = back_to_back(TILED[name][0])
    plan = planned(name, "bf16", weight)
    out = torch.full((n,), 7.0, device=DEV, dtype=T[weight])
    B.ar_orthogonalize(plan, torch.zeros(n, device=DEV, dtype=torch.bfloat16), out)
    torch.cuda.synchronize()
    assert (out == 0).all()
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("name", ["small", "mixed", "square"])
def test_in_place_and_the_same_bits_every_time(name, dtype):
    shapes = TILED[name][0]
    offs, n = back_to_back(shapes)
    g = arena(matrices(shapes, "normal", 8), offs, n, dtype)
    plan = planned(name, dtype, dtype)
    outs = [torch.empty_like(g) for _ in range(3)]
    for out in outs:
        B.ar_orthogonalize(plan, g, out)
    B.ar_orthogonalize(plan, g, g)
    torch.cuda.synchronize()
    assert all(torch.equal(g, out) for out in outs)
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["small", "mixed", "large"])
def test_graph_replays(name):
    """A captured step replayed between eager steps, against fp64 as well."""
    shapes = TILED[name][0]
    offs, n = back_to_back(shapes)
    plan = planned(name, "bf16", "fp32")
    B.ar_muon_plan_prepare(plan)
    g, m, w = torch.empty(n, device=DEV, dtype=torch.bfloat16), torch.zeros(n, device=DEV), torch.randn(n, device=DEV)
    m2, w2 = m.clone(), w.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.ar_muon_step(plan, g, m, w, 0.1, weight_decay=0.1, stream=s)
    for _ in range(3):
        g.normal_()
        before, mom = w.clone(), m.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        B.ar_muon_step(plan, g, m2, w2, 0.1, weight_decay=0.1)
        torch.cuda.synchronize()
        assert torch.equal(m, m2) and torch.equal(w, w2)
    (r, c), part = shapes[0], slice(0, shapes[0][0] * shapes[0][1])
    u = g[part].double() * 1.95 + 0.95 ** 2 * mom[part].double()
    o, scale = orthogonalized(u.view(r, c), [COEF] * 5), math.sqrt(max(1, r / c))
    want = 0.99 * before[part].double().view(r, c) - 0.1 * scale * o
    tol = 0.1 * scale * tolerance(o, "fp32") * float(o.norm()) + 5 * 2.0 ** -24 * float(want.norm())
    assert float((w[part].view(r, c).double() - want).norm()) <= tol
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["small", "mixed"])
def test_arena_past_32_bits(name):
    shapes = TILED[name][0]
    offs = [((1 << 32) + 5 if i else 1) + (i << 24) for i in range(len(shapes))]
    n = offs[-1] + shapes[-1][0] * shapes[-1][1]
    plan = planned(name, "bf16", "bf16", offs)
    g = torch.zeros(n, device=DEV, dtype=torch.bfloat16)
    for (r, c), o in zip(shapes, offs):
        g[o:o + r * c].normal_()
    out = torch.empty_like(g)
    B.ar_orthogonalize(plan, g, out)
    torch.cuda.synchronize()
    for (r, c), o in zip(shapes, offs):
        want = orthogonalized(g[o:o + r * c].view(r, c), [COEF] * 5)
        check(out[o:o + r * c].view(r, c), want, tolerance(want, "bf16"), f"{r}x{c}")
    B.ar_muon_plan_destroy(plan)


@pytest.mark.gpu
def test_experts_reduce_then_step():
    """Expert weight gradients into every rank's bucketed arena, the all-reduce, and a tiled Muon step of it."""
    ranks, e, inf, outf, tokens = 3, 2, 224, 352, 300
    bp = B.ar_bucket_plan_create(ranks, 1, [inf * outf] * e, "fp32", "ring", 2 * inf * outf * 4)
    offs, count = B.ar_bucket_layout(bp, e)
    ex = B.ar_experts_create(e, inf, outf, "bf16", "fp32", offs)
    mu = B.ar_muon_plan_create([(outf, inf)] * e, "fp32", "fp32", offs)
    assert B.ar_muon_plan_stats(mu)["launches"] > 1
    arenas = [torch.zeros(count, device=DEV) for _ in range(ranks)]
    w, m = torch.randn(count, device=DEV), torch.zeros(count, device=DEV)
    w0 = w.clone()
    rng, want = np.random.default_rng(4), [torch.zeros(outf, inf, dtype=torch.float64, device=DEV) for _ in range(e)]
    for a in arenas:
        x, dy = (torch.randn(tokens, f, device=DEV).bfloat16() for f in (inf, outf))
        cut = int(rng.integers(0, tokens + 1))
        ends = torch.tensor([cut, tokens], dtype=torch.int32, device=DEV)
        for k, rows in enumerate((slice(0, cut), slice(cut, tokens))):
            want[k] += dy[rows].double().t().contiguous() @ x[rows].double()
        B.ar_experts_weight_grad(ex, x, dy, a, ends)
    B.ar_bucket_allreduce(bp, arenas, torch.cuda.current_stream())
    B.ar_muon_step(mu, arenas[1], m, w, 0.1, mu=0.0, grad_scale=1 / ranks, nesterov=False)
    torch.cuda.synchronize()
    for k in range(e):
        part, scale = slice(offs[k], offs[k] + inf * outf), math.sqrt(outf / inf)
        # the step against the arena that it read
        o = orthogonalized(arenas[1][part].double().view(outf, inf) / ranks, [COEF] * 5)
        wd = w0[part].view(outf, inf).double() - 0.1 * scale * o
        tol = 0.1 * scale * tolerance(o, "fp32") * float(o.norm()) + 5 * 2.0 ** -24 * float(wd.norm())
        assert float((w[part].view(outf, inf).double() - wd).norm()) <= tol
        for a in arenas:  # sums of `tokens` products per rank and of the ranks, in fp32
            assert float((a[part].view(outf, inf).double() - want[k]).norm()) <= 2.0 ** -18 * float(want[k].norm())
    B.ar_bucket_plan_destroy(bp)
    B.ar_experts_destroy(ex)
    B.ar_muon_plan_destroy(mu)
