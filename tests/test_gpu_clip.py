"""The global gradient norm and clipping against a plain fp64 implementation,
on cuda:0.

Tolerances.  Squares and sums are fp64 (n elements: n 2^-53), the norm is
rounded once to fp32: 2^-24, and 2^-30 for the rest.  The factor takes the
norm's error and one rounding to fp32, the product one in fp32 and one to the
gradients' type (half a step of finfo(t).eps / 2).
"""
import math

import pytest
import torch

from gradient_all_reduce_ar_amd import _binding as B

DEV = "cuda:0"
T = {"fp32": torch.float32, "bf16": torch.bfloat16}
NORM_TOL = 2.0 ** -24 + 2.0 ** -30


class Case:
    def __init__(self, counts, dtype, offsets=None, shift=0, sigma=1e-3, seed=0, extra=5):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        at, self.offsets = 0, []
        for n in counts:
            self.offsets.append(at)
            at += n
        if offsets:
            self.offsets = offsets
        self.counts, self.dtype = counts, dtype
        self.size = max([o + n for o, n in zip(self.offsets, counts)] + [0]) + extra
        self.grads = torch.randn(self.size + shift, generator=g, device=DEV).mul_(sigma).to(T[dtype])[shift:]
        self.held = torch.zeros(self.size, dtype=torch.bool, device=DEV)
        for o, n in zip(self.offsets, counts):
            self.held[o:o + n] = True
        self.grads[~self.held] = 1e30  # what lies between would be seen
        self.plan = B.ar_norm_plan_create(counts, dtype, self.offsets)
        self.norm = torch.full((1,), -1.0, device=DEV)
        self.each = torch.full((max(1, len(counts)),), -1.0, device=DEV)

    def want(self, g=None):
        g = self.grads if g is None else g
        return torch.stack([g[o:o + n].double().square().sum() for o, n in zip(self.offsets, self.counts)]
                           + [torch.zeros((), dtype=torch.float64, device=DEV)])[:-1]

    def check_norm(self, scale=1.0):
        squares = self.want()
        assert abs(float(self.norm) - scale * math.sqrt(float(squares.sum()))) <= NORM_TOL * scale * math.sqrt(float(squares.sum())) + 1e-45
        want = scale * squares.sqrt()
        got = self.each[:len(self.counts)].double()
        assert ((got - want).abs() <= NORM_TOL * want + 1e-45).all()

    def check_clip(self, out, before, most):
        norm = math.sqrt(float(self.want(before).sum()))
        c = min(1.0, most / (norm + 1e-6))
        want = before.double() * c
        tol = (3 * 2.0 ** -24 + torch.finfo(T[self.dtype]).eps / 2) * (1 + 2.0 ** -7) * want.abs() + 1e-40
        bad = ((out.double() - want).abs() > tol) & self.held
        assert not bad.any(), int(bad.sum())


LISTS = [
    [1], [0], [], [7], [8], [9], [511, 1, 513], [64 * 64] * 4, [3, 0, 5, 0, 1], [1000] * 70, [1] * 5000,
    [100003, 5, 77777, 1], [1 << 20, 12345], [5000003], [2, 16 << 20],
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("counts", LISTS, ids=lambda c: f"{len(c)}-{sum(c)}")
def test_norm_and_clip(counts, dtype, shift):
    print("case", len(counts), sum(counts), dtype, shift, flush=True)
    c = Case(counts, dtype, shift=shift)
    B.ar_grad_norm(c.plan, c.grads, c.norm, c.each)
    torch.cuda.synchronize()
    c.check_norm()
    alone = torch.full((1,), -1.0, device=DEV)
    B.ar_grad_norm(c.plan, c.grads, alone, scale=0.25)
    B.ar_grad_norm(c.plan, c.grads, c.norm)
    torch.cuda.synchronize()
    assert float(alone) == 0.25 * float(c.norm)  # a power of two: the same number
    before = c.grads.clone()
    for most in (0.5 * float(c.norm) + 1e-9, 2.0 * float(c.norm) + 1.0):
        out = torch.full((c.size + 2,), 7.0, device=DEV, dtype=T[dtype])[2:]  # lies otherwise than grads
        B.ar_grad_clip(c.plan, c.grads, c.norm, most, out)
        torch.cuda.synchronize()
        assert torch.equal(c.grads, before)
        c.check_clip(out, before, most)
        assert (out[~c.held] == 7).all(), "elements between the tensors changed"
    B.ar_grad_clip(c.plan, c.grads, c.norm, 2.0 * float(c.norm) + 1.0)  # in place, nothing to do
    torch.cuda.synchronize()
    assert torch.equal(c.grads, before)
    most = 0.5 * float(c.norm) + 1e-9
    B.ar_grad_clip(c.plan, c.grads, c.norm, most)
    torch.cuda.synchronize()
    c.check_clip(c.grads, before, most)
    assert torch.equal(c.grads[~c.held], before[~c.held])
    B.ar_norm_plan_destroy(c.plan)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_gaps_and_orders(dtype):
    """Tensors in any order, off every alignment, with gaps."""
    c = Case([1000, 17, 40000, 0, 1], dtype, offsets=[50001, 3, 5003, 0, 1])
    B.ar_grad_norm(c.plan, c.grads, c.norm, c.each)
    torch.cuda.synchronize()
    c.check_norm()
    out = torch.full_like(c.grads, 7.0)
    B.ar_grad_clip(c.plan, c.grads, c.norm, 1e-3, out)
    torch.cuda.synchronize()
    c.check_clip(out, c.grads, 1e-3)
    assert (out[~c.held] == 7).all()
    B.ar_norm_plan_destroy(c.plan)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("sigma", [1e-42, 1e-30, 1e25, 1e35])
def test_any_size(dtype, sigma):
    """Squares that fp32 does not hold."""
    c = Case([5000, 3000], dtype, sigma=sigma)
    c.grads[~c.held] = 0
    B.ar_grad_norm(c.plan, c.grads, c.norm, c.each)
    torch.cuda.synchronize()
    squares = c.want()
    norm = math.sqrt(float(squares.sum()))
    assert abs(float(c.norm) - norm) <= NORM_TOL * norm + 2.0 ** -149  # (a denormal norm: one step)
    out = torch.empty_like(c.grads)
    B.ar_grad_clip(c.plan, c.grads, c.norm, 1.0, out)
    torch.cuda.synchronize()
    c.check_clip(out, c.grads, 1.0)
    B.ar_norm_plan_destroy(c.plan)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_not_finite(dtype, value):
    """An infinite norm takes every gradient to zero and the infinity to NaN; a NaN norm takes all to NaN."""
    c = Case([5000, 300, 9], dtype)
    c.grads[5100] = value
    B.ar_grad_norm(c.plan, c.grads, c.norm, c.each)
    out = torch.full_like(c.grads, 7.0)
    B.ar_grad_clip(c.plan, c.grads, c.norm, 1.0, out)
    torch.cuda.synchronize()
    want = abs(value)
    assert math.isnan(float(c.norm)) if math.isnan(want) else float(c.norm) == want
    each = c.each.tolist()
    assert math.isfinite(each[0]) and math.isfinite(each[2]) and not math.isfinite(each[1])
    if math.isnan(want):
        assert out[c.held].isnan().all()
    else:
        ref = (c.grads.float() * 0.0).to(out.dtype)
        assert torch.equal(out[c.held].isnan(), ref[c.held].isnan()) and (out[c.held].nan_to_num(0) == 0).all()
    B.ar_norm_plan_destroy(c.plan)


@pytest.mark.gpu
def test_joined_norm():
    """The norm of two arenas, joined on the device, clips both."""
    a, b = Case([5000], "fp32", seed=1), Case([70000, 3], "bf16", seed=2)
    B.ar_grad_norm(a.plan, a.grads, a.norm)
    B.ar_grad_norm(b.plan, b.grads, b.norm)
    norm = (a.norm.double().square() + b.norm.double().square()).sqrt().float()
    most = 0.01
    for c in (a, b):
        out = torch.empty_like(c.grads)
        B.ar_grad_clip(c.plan, c.grads, norm, most, out)
        want = c.grads.double() * min(1.0, most / (float(norm) + 1e-6))
        tol = (2 * 2.0 ** -24 + torch.finfo(out.dtype).eps / 2) * (1 + 2.0 ** -7) * want.abs() + 1e-40
        assert (((out.double() - want).abs() <= tol) | ~c.held).all()
        B.ar_norm_plan_destroy(c.plan)


@pytest.mark.gpu
def test_repeats_and_streams():
    """The same bits every time, on any stream, whatever ran before; two plans at once."""
    a, b = Case([300000, 17, 70001], "bf16", seed=3), Case([200001] * 3, "fp32", seed=4)
    for c in (a, b):
        B.ar_grad_norm(c.plan, c.grads, c.norm, c.each)
    torch.cuda.synchronize()
    want = [(c.norm.clone(), c.each.clone()) for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for c, s in zip((a, b), streams):
            c.norm.fill_(-1)
            c.each.fill_(-1)
            s.wait_stream(torch.cuda.current_stream())
            B.ar_grad_norm(c.plan, c.grads, c.norm, c.each, stream=s)
        torch.cuda.synchronize()
        for c, (n, e) in zip((a, b), want):
            assert torch.equal(c.norm, n) and torch.equal(c.each, e)
    for c in (a, b):
        B.ar_norm_plan_destroy(c.plan)


@pytest.mark.gpu
def test_captured():
    """Norm and clip in a graph, replayed on changing gradients with eager calls between; a capture of a plan that
    is not prepared is refused."""
    c = Case([300000, 17, 70001], "bf16", seed=5)
    out = torch.zeros_like(c.grads)
    graph = torch.cuda.CUDAGraph()
    B.ar_norm_plan_prepare(c.plan)
    other = B.ar_norm_plan_create([10], "fp32")
    with torch.cuda.graph(graph):
        s = torch.cuda.current_stream()
        B.ar_grad_norm(c.plan, c.grads, c.norm, c.each, stream=s)
        B.ar_grad_clip(c.plan, c.grads, c.norm, 0.1, out, stream=s)
        with pytest.raises(ValueError, match="prepared"):
            B.ar_grad_norm(other, torch.empty(10, device=DEV), c.norm, stream=s)
    for k in range(4):
        c.grads[c.held] = (torch.randn(int(c.held.sum()), device=DEV) * 10.0 ** -k).bfloat16()
        graph.replay()
        torch.cuda.synchronize()
        got, each, clipped = c.norm.clone(), c.each.clone(), out.clone()
        c.check_norm()
        c.check_clip(out, c.grads, 0.1)
        B.ar_grad_norm(c.plan, c.grads, c.norm, c.each)
        B.ar_grad_clip(c.plan, c.grads, c.norm, 0.1, out)
        torch.cuda.synchronize()
        assert torch.equal(got, c.norm) and torch.equal(each, c.each) and torch.equal(clipped[c.held], out[c.held])
    B.ar_norm_plan_destroy(other)
    B.ar_norm_plan_destroy(c.plan)


@pytest.mark.gpu
def test_far_offsets():
    """Elements past 2^31 (bytes past 2^32)."""
    at = (1 << 31) + 5
    g = torch.zeros(at + 70000, device=DEV, dtype=torch.bfloat16)
    g[at:at + 65537] = 0.5
    g[11:111] = 2.0
    plan = B.ar_norm_plan_create([65537, 100], "bf16", [at, 11])
    norm = torch.zeros(1, device=DEV)
    B.ar_grad_norm(plan, g, norm)
    B.ar_grad_clip(plan, g, norm, 1.0)
    torch.cuda.synchronize()
    want = math.sqrt(65537 * 0.25 + 400)
    assert abs(float(norm) - want) <= NORM_TOL * want
    c = 1 / (want + 1e-6)
    assert ((g[at:at + 65537].double() - 0.5 * c).abs() <= 2.0 ** -8 * 0.5 * c).all()
    assert ((g[11:111].double() - 2 * c).abs() <= 2.0 ** -8 * 2 * c).all()
    assert float(g[at + 65537:].abs().max()) == 0 and float(g[111:1 << 20].abs().max()) == 0
    B.ar_norm_plan_destroy(plan)


@pytest.mark.gpu
def test_tensor_checks():
    c = Case([64], "bf16")
    for bad, word in ((c.grads.float(), "wanted"), (c.grads[:32], "holds"), (c.grads.cpu(), "device tensor")):
        with pytest.raises(ValueError, match=word):
            B.ar_grad_norm(c.plan, bad, c.norm)
    with pytest.raises(ValueError, match="wanted"):
        B.ar_grad_norm(c.plan, c.grads, c.norm.double())
    with pytest.raises(ValueError, match="holds"):
        B.ar_grad_norm(c.plan, c.grads, c.norm, c.each[:0])
    B.ar_norm_plan_destroy(c.plan)


def near_a_tie(dtype):
    """Gradients whose squares add up to hardly more than the middle between two fp32 norms: a chunk's worth of small
    ones with a large one behind them, which take the norm to the other side where they are added to it one by one.
    (Counts so that a chunk of the plan is an eighth of them, a wave's work.)"""
    n, lost = {"fp32": (16384, 16), "bf16": (32768, 32)}[dtype]
    chunk, small, middle = n // 8, 2.0 ** -3, (1 << 24) + 1
    g = torch.zeros(n, dtype=torch.float64)
    g[:chunk - 1], g[chunk - 1] = small, 2.0 ** 24
    rest = middle ** 2 + lost / 2 * small ** 2 - float(g.square().sum())  # in other chunks
    at = 2 * chunk
    while rest >= 1:
        v = torch.tensor(math.floor(math.sqrt(rest))).to(T[dtype])
        if float(v) ** 2 > rest:
            v = torch.nextafter(v, torch.zeros_like(v))
        g[at] = float(v)
        rest, at = rest - float(v) ** 2, at + 3
    left = int(rest / small ** 2)
    g[3 * chunk:3 * chunk + left] = small
    assert float(g.square().sum()) == middle ** 2 + lost / 2 * small ** 2 and torch.equal(g.to(T[dtype]).double(), g)
    return g.to(T[dtype])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_norm_is_the_same_at_any_address(dtype):
    """The order of the sums is the plan's: the same gradients have the same norm wherever their arena lies."""
    g = near_a_tie(dtype)
    n = g.numel()
    plan = B.ar_norm_plan_create([n], dtype)
    got = []
    for shift in range(8):
        arena = torch.zeros(n + 8, device=DEV, dtype=T[dtype])
        arena[shift:shift + n] = g.to(DEV)
        norm, each = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
        B.ar_grad_norm(plan, arena[shift:shift + n], norm, each)
        torch.cuda.synchronize()
        got.append((float(norm), float(each)))
    assert len(set(got)) == 1, got
    assert abs(got[0][0] - ((1 << 24) + 1)) <= 1  # either neighbour of the middle
    B.ar_norm_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_norm_beyond_fp32(dtype):
    """Finite gradients whose norm fp32 does not hold: infinite, and so c = 0; with a scale that it holds, the norm."""
    g = torch.full((5000,), 3e38, device=DEV).to(T[dtype])
    plan = B.ar_norm_plan_create([4999, 1], dtype)
    norm, each, out = torch.zeros(1, device=DEV), torch.zeros(2, device=DEV), torch.empty_like(g)
    B.ar_grad_norm(plan, g, norm, each)
    B.ar_grad_clip(plan, g, norm, 1.0, out)
    torch.cuda.synchronize()
    assert float(norm) == float("inf") and each.tolist() == [float("inf"), float(g[0])] and (out == 0).all()
    B.ar_grad_norm(plan, g, norm, scale=2.0 ** -10)
    torch.cuda.synchronize()
    want = 2.0 ** -10 * math.sqrt(5000) * float(g[0])
    assert abs(float(norm) - want) <= NORM_TOL * want
    B.ar_norm_plan_destroy(plan)
