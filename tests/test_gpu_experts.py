"""The expert products against a plain fp64 implementation, on cuda:0.

Tolerance of an element.  A product of two bf16 numbers is exact in fp32, one
of two fp32 numbers is off by half a step (2^-24); a sum of k of them in fp32,
in any order, is off by at most k steps of 2^-23 (whether the adder rounds or
cuts) of the sum of their magnitudes.  The result is then rounded once to its
type (half a step: finfo(t).eps / 2 of the value).
"""
import numpy as np
import pytest
import torch

from gradient_all_reduce_ar_amd import _binding as B
from tests.test_operators_cpu import ROWS_OF_DISPATCH, OnDevice, launch_shapes

DEV = "cuda:0"
T = {"fp32": torch.float32, "bf16": torch.bfloat16}


def close(got, want, mag, k, what):
    """|got - want| within the tolerance above, element by element."""
    half = torch.finfo(got.dtype).eps / 2
    tol = (k + 2) * 2.0 ** -23 * mag + half * want.abs() * (1 + 2.0 ** -7) + 1e-37
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} elements off, worst {float((off / tol).nan_to_num(0).max()):.3g} tolerances"


class Case:
    def __init__(self, inf, outf, counts, dtype, grad="fp32", extra=0, seed=0, pad=(0, 0), shift=0, offsets=None):
        self.counts, self.inf, self.outf, self.dtype, self.grad = counts, inf, outf, dtype, grad
        self.t = sum(counts) + extra
        e = len(counts)
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.offsets = offsets
        size = inf * outf
        self.at = offsets or [k * size for k in range(e)]
        self.arena = max(self.at) + size
        self.x = self.rows(inf, pad[0], shift, g)
        self.dy = self.rows(outf, pad[1], shift, g)
        self.w = torch.randn(self.arena + shift, generator=g, device=DEV).to(T[dtype])[shift:]
        self.ends = torch.from_numpy(np.cumsum(counts).astype(np.int32)).to(DEV)
        self.plan = B.ar_experts_create(e, inf, outf, dtype, grad, offsets)
        self.pad, self.shift = pad, shift

    def rows(self, n, pad, shift, g=None):
        """[t, n] with a row stride of n + pad, `shift` elements into its storage; random, or all 7."""
        flat = torch.full((self.t * (n + pad) + shift,), 7.0, device=DEV)
        if g is not None:
            flat.normal_(generator=g)
        return flat.to(T[self.dtype])[shift:].view(self.t, n + pad)[:, :n]

    def weight(self, e):
        return self.w[self.at[e]:self.at[e] + self.inf * self.outf].view(self.outf, self.inf)

    def groups(self):
        lo = 0
        for e, n in enumerate(self.counts):
            yield e, slice(lo, lo + n)
            lo += n

    def check_rows(self, y, src, grad):
        assert (y[sum(self.counts):].double() == 7).all(), "rows behind the last expert changed"
        for e, s in self.groups():
            a, w = src[s].double(), self.weight(e).double()
            b = w if grad else w.t().contiguous()
            close(y[s], a @ b, a.abs() @ b.abs(), b.shape[0], f"expert {e}")

    def forward(self, stream=None):
        y = self.rows(self.outf, self.pad[1], self.shift)
        B.ar_experts_forward(self.plan, self.x, self.w, y, self.ends, stream)
        return y

    def input_grad(self, stream=None):
        dx = self.rows(self.inf, self.pad[0], self.shift)
        B.ar_experts_input_grad(self.plan, self.dy, self.w, dx, self.ends, stream)
        return dx

    def weight_grad(self, accumulate=False):
        g = torch.full((self.arena + self.shift,), 3.0, device=DEV, dtype=T[self.grad])[self.shift:]
        B.ar_experts_weight_grad(self.plan, self.x, self.dy, g, self.ends, accumulate)
        return g

    def check_weights(self, g, accumulate=False):
        held = torch.zeros(self.arena, dtype=torch.bool, device=DEV)
        for e, s in self.groups():
            part = slice(self.at[e], self.at[e] + self.inf * self.outf)
            held[part] = True
            dyt, x = self.dy[s].double().t().contiguous(), self.x[s].double().contiguous()
            want, mag = dyt @ x, dyt.abs() @ x.abs()
            if accumulate:
                want, mag = want + 3, mag + 3
            close(g[part].view(self.outf, self.inf), want, mag, dyt.shape[1] + 1, f"expert {e}")
        assert ((g[:self.arena] == 3) | held).all(), "the arena changed outside the matrices"

    def check_all(self):
        y, dx, g, g2 = self.forward(), self.input_grad(), self.weight_grad(), self.weight_grad(True)
        torch.cuda.synchronize()
        self.check_rows(y, self.x, False)
        self.check_rows(dx, self.dy, True)
        self.check_weights(g)
        self.check_weights(g2, True)
        B.ar_experts_destroy(self.plan)


SIZES = [
    # in, out, rows of each expert
    (64, 64, [1]), (64, 64, [0, 0, 1]), (8, 8, [3, 0, 2]), (1, 1, [5, 2]), (1, 40, [5, 2]), (40, 1, [5, 2]),
    (64, 128, [128, 128]), (128, 64, [127, 129, 1, 0]), (72, 136, [33, 0, 65, 200]), (200, 264, [31, 32, 33]),
    (71, 135, [5, 0, 200, 300, 1]), (129, 257, [130, 64]), (66, 34, [17, 100]), (512, 1024, [500, 800, 1, 700]),
    (1000, 520, [3, 2, 1, 1]), (320, 192, [16, 15, 17, 1, 0, 2]), (136, 72, list(range(70))),
    (64, 64, [0] * 64 + [1] + [0] * 64 + [7]), (2048, 64, [2, 1]), (64, 2048, [1, 1, 1]), (264, 640, [700]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,grad", [("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("inf,outf,counts", SIZES, ids=[f"{i}x{o}-{len(c)}e-{sum(c)}" for i, o, c in SIZES])
def test_products(inf, outf, counts, dtype, grad):
    print("case", inf, outf, counts, dtype, grad, flush=True)
    Case(inf, outf, counts, dtype, grad, extra=3).check_all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,grad", [("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("inf,outf,counts", [(128, 64, [4000]), (72, 136, [2100, 0, 700]), (71, 135, [3001, 5]),
                                             (512, 768, [8001]), (64, 64, [0, 0, 0, 4099, 1])])
def test_long_weight_gradients(inf, outf, counts, dtype, grad):
    """Few tiles and many rows: the rows are cut into parts and joined; experts of none, one and many rows."""
    print("case", inf, outf, counts, dtype, grad, flush=True)
    Case(inf, outf, counts, dtype, grad, extra=3).check_all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,grad", [("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("inf,outf,counts", [(2048, 2056, [300, 724, 0, 77]), (1031, 1029, [300, 400, 0, 500]),
                                             (2056, 4104, [2100]), (1000, 4000, [513, 1500, 1])])
def test_large_tiles(inf, outf, counts, dtype, grad):
    """Sizes that the larger tiles are for, with edges in every direction."""
    print("case", inf, outf, counts, dtype, grad, flush=True)
    Case(inf, outf, counts, dtype, grad, extra=5).check_all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("inf,outf", [(1, 1), (3, 2), (7, 5), (2, 131), (129, 3), (257, 263), (1031, 67)])
@pytest.mark.parametrize("counts", [[70, 0, 65, 1], [300, 129, 64, 2]])
def test_narrow_and_odd_rows(inf, outf, counts, dtype):
    """Rows of a few elements, and tiles whose last columns end inside a load, over several stages; what lies
    behind the last row and in the gaps is NaN."""
    print("case", inf, outf, counts, dtype, flush=True)
    c = Case(inf, outf, counts, dtype, extra=2)
    c.x[sum(counts):], c.dy[sum(counts):] = float("nan"), float("nan")
    c.check_all()
    c = Case(inf, outf, counts, dtype, extra=2, pad=(1, 2))
    for t, n, pad in ((c.x, inf, 1), (c.dy, outf, 2)):
        t.as_strided((c.t, n + pad), (n + pad, 1))[:, n:] = float("nan")
    c.check_all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,shift", [((8, 16), 0), ((1, 3), 0), ((0, 0), 1), ((8, 8), 3), ((5, 0), 8), ((4, 4), 4)])
def test_strides_and_alignment(pad, shift, dtype):
    """Rows with gaps, and rows, weights and gradients that start off 16 bytes; the gaps stay as they were."""
    print("case", pad, shift, dtype, flush=True)
    c = Case(64, 136, [40, 0, 133], dtype, extra=2, pad=pad, shift=shift)
    y = c.forward()
    torch.cuda.synchronize()
    full = y.as_strided((c.t, c.outf + pad[1]), (c.outf + pad[1], 1))
    assert (full[:, c.outf:].double() == 7).all(), "the gap between rows changed"
    c.check_all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_weight_offsets(dtype):
    """Matrices in any order, with gaps, at odd elements."""
    size = 40 * 24
    for offs in ([2 * size + 64, 0, 4 * size], [2 * size + 7, 1, 4 * size + 3]):
        Case(40, 24, [9, 50, 3], dtype, offsets=offs).check_all()


@pytest.mark.gpu
@pytest.mark.parametrize("ends,want", [
    ([5, 3, 9], [(0, 5), (5, 5), (5, 9)]), ([-4, 6, 6], [(0, 0), (0, 6), (6, 6)]),
    ([4, 1 << 30, 2], [(0, 4), (4, 12), (12, 12)]), ([-1, -(1 << 31), -7], [(0, 0)] * 3), ([0, 0, 0], [(0, 0)] * 3),
])
def test_ends_are_clamped(ends, want):
    """Any contents of ends are a running maximum inside [0, tokens]."""
    c = Case(64, 64, [4, 4, 4], "bf16")
    c.ends = torch.tensor(ends, dtype=torch.int32, device=DEV)
    c.counts = [b - a for a, b in want]
    c.check_all()


@pytest.mark.gpu
def test_no_tokens():
    c = Case(64, 64, [0, 0], "bf16")
    e = torch.empty(0, 64, device=DEV, dtype=torch.bfloat16)
    g = torch.full((2 * 64 * 64,), 3.0, device=DEV)
    B.ar_experts_forward(c.plan, e, c.w, e, c.ends)
    B.ar_experts_weight_grad(c.plan, e, e, g, c.ends, accumulate=True)
    torch.cuda.synchronize()
    assert (g == 3).all()
    B.ar_experts_weight_grad(c.plan, e, e, g, c.ends)
    torch.cuda.synchronize()
    assert (g == 0).all()
    B.ar_experts_destroy(c.plan)


@pytest.mark.gpu
@pytest.mark.parametrize("inf,dtype", [(64, "bf16"), (71, "bf16"), (512, "bf16"), (64, "fp32")])
@pytest.mark.parametrize("rows", [40, 200])
def test_infinities_stay_in_their_rows(inf, dtype, rows):
    """An infinity or NaN in one row of x changes that row of y alone; one in an expert's rows changes that
    expert's gradient alone; rows behind the last expert and a row's padding may hold anything."""
    c = Case(inf, 72, [rows, rows], dtype, extra=4, pad=(8, 8))
    clean, gclean = c.forward(), c.weight_grad()
    c.x.as_strided((c.t, inf + 8), (inf + 8, 1))[:, inf:] = float("nan")
    c.x[2 * rows:] = float("nan")
    c.dy[2 * rows:] = float("inf")
    c.x[3] = float("nan")
    c.x[rows - 1, 0] = float("inf")
    y, g = c.forward(), c.weight_grad()
    torch.cuda.synchronize()
    keep = torch.ones(2 * rows, dtype=torch.bool, device=DEV)
    keep[3] = keep[rows - 1] = False
    assert torch.equal(y[:2 * rows][keep], clean[:2 * rows][keep])
    assert y[3].isnan().all() and not y[rows - 1].isfinite().any()
    size = inf * 72
    assert torch.equal(g[size:], gclean[size:]) and g[:size].isnan().all()
    B.ar_experts_destroy(c.plan)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[1, 2, 0, 1], [100, 300, 0, 77], [1000, 3000, 0, 700]])
def test_graph_replays(counts):
    """A captured forward, input gradient and weight gradient, replayed with new rows and new ends between
    eager calls."""
    c = Case(128, 256, counts, "bf16", extra=8)
    B.ar_experts_prepare(c.plan)
    y, dx = c.rows(256, 0, 0), c.rows(128, 0, 0)
    g = torch.empty(c.arena, device=DEV)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.ar_experts_forward(c.plan, c.x, c.w, y, c.ends, s)
        B.ar_experts_input_grad(c.plan, c.dy, c.w, dx, c.ends, s)
        B.ar_experts_weight_grad(c.plan, c.x, c.dy, g, c.ends, stream=s)
    for k in range(4):
        c.x.normal_()
        c.dy.normal_()
        c.counts = c.counts[1:] + c.counts[:1]
        c.ends.copy_(torch.from_numpy(np.cumsum(c.counts).astype(np.int32)))
        y.fill_(7)
        dx.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, c.forward()) and torch.equal(dx, c.input_grad())
        assert torch.equal(g, c.weight_grad())
        c.check_rows(y, c.x, False)
    B.ar_experts_destroy(c.plan)


@pytest.mark.gpu
@pytest.mark.parametrize("address", [False, True])
def test_capture_needs_a_prepared_plan(address):
    c = Case(64, 32, [5, 0, 20], "bf16")
    y, other = c.rows(32, 0, 0), torch.zeros(4, device=DEV)
    t = [c.x, c.w, y, c.ends]
    if address:
        t, more = [v.data_ptr() for v in t], dict(ntokens=c.x.shape[0], x_stride=c.x.stride(0), y_stride=y.stride(0))
    else:
        more = {}
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        with pytest.raises(B.ArError if address else ValueError):
            B.ar_experts_forward(c.plan, *t, stream=s, **more)
        other.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert other.tolist() == [1] * 4 and B.ar_experts_stats(c.plan)["device"] == -1
    B.ar_experts_forward(c.plan, *t, **more)
    torch.cuda.synchronize()
    c.check_rows(y, c.x, False)
    B.ar_experts_destroy(c.plan)


@pytest.mark.gpu
def test_two_streams_at_once():
    """One plan's calls have no workspace: two streams may run them together."""
    c = Case(256, 512, [700, 100, 0, 900], "bf16")
    want, wantx = c.forward(), c.input_grad()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [c.rows(512, 0, 0) for _ in range(6)] + [c.rows(256, 0, 0) for _ in range(6)]
    torch.cuda.synchronize()
    for i in range(6):
        B.ar_experts_forward(c.plan, c.x, c.w, outs[i], c.ends, a)
        B.ar_experts_input_grad(c.plan, c.dy, c.w, outs[6 + i], c.ends, b)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs[:6]) and all(torch.equal(o, wantx) for o in outs[6:])
    B.ar_experts_destroy(c.plan)


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1])
def test_arena_past_32_bits(shift):
    """A matrix that starts past 2^32 elements."""
    at = (1 << 32) + 4096 + shift
    c = Case(64, 72, [20, 150], "bf16", "bf16", offsets=[shift, at])
    c.check_all()


@pytest.mark.gpu
def test_rows_past_32_bits():
    """Rows whose elements lie past 2^32 (a row stride of 2^22)."""
    t, stride = 1100, 1 << 22
    x = torch.zeros(t * stride, device=DEV, dtype=torch.bfloat16).view(t, stride)[:, :64]
    x.normal_()
    c = Case(64, 72, [500, 600], "bf16")
    y = torch.empty(t, 72, device=DEV, dtype=torch.bfloat16)
    B.ar_experts_forward(c.plan, x, c.w, y, c.ends)
    c.x = x
    g = c.weight_grad()
    torch.cuda.synchronize()
    c.check_rows(y, x, False)
    c.check_weights(g)
    B.ar_experts_destroy(c.plan)


@pytest.mark.gpu
def test_gradients_against_differences():
    """input_grad and weight_grad are the derivatives of forward: with the loss sum(dy * y), which is linear in
    x and in W, a difference of losses is the gradient's inner product up to the roundings of fp32."""
    c = Case(48, 40, [7, 0, 21], "fp32")
    dx, g = c.input_grad(), c.weight_grad()
    y0 = c.forward().double()
    step = torch.randn_like(c.x)
    c.x += step
    y1 = c.forward().double()
    c.x -= step
    moved = ((y1 - y0) * c.dy.double()).sum()
    along = (dx.double() * step.double()).sum()
    size = float((dx.double() * step.double()).abs().sum() + (y1.abs() * c.dy.double().abs()).sum())
    assert abs(float(moved - along)) <= 64 * 2.0 ** -23 * size
    wstep = torch.randn_like(c.w)
    c.w += wstep
    y2 = c.forward().double()
    moved, along = ((y2 - y0) * c.dy.double()).sum(), (g.double() * wstep.double()).sum()
    size = float((g.double() * wstep.double()).abs().sum() + (y2.abs() * c.dy.double().abs()).sum())
    assert abs(float(moved - along)) <= 64 * 2.0 ** -23 * size
    B.ar_experts_destroy(c.plan)


@pytest.mark.gpu
def test_refusals_on_the_device():
    c = Case(64, 72, [3, 4], "bf16")
    y = torch.empty(7, 72, device=DEV, dtype=torch.bfloat16)
    for bad in (dict(x=c.x[:, :32]), dict(x=c.x.float()), dict(x=c.x.t()), dict(y=y[:5]), dict(w=c.w[:-1]),
                dict(ends=c.ends[:1]), dict(ends=c.ends.long()), dict(ends=c.ends.float())):
        a = dict(x=c.x, w=c.w, y=y, ends=c.ends) | bad
        with pytest.raises(ValueError):
            B.ar_experts_forward(c.plan, a["x"], a["w"], a["y"], a["ends"])
    B.ar_experts_destroy(c.plan)


def ragged(experts, tokens, seed=0):
    """Rows of each expert: some none, some one, the rest uneven."""
    rng = np.random.default_rng(seed)
    share = rng.dirichlet(np.full(experts, 0.7))
    counts = np.floor(share * tokens).astype(np.int64)
    counts[int(rng.integers(experts))] += tokens - counts.sum()
    return [int(c) for c in counts]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,inf,outf,experts,tokens,forward,input_grad,weight_grad,parts", ROWS_OF_DISPATCH)
def test_every_tile(dtype, inf, outf, experts, tokens, forward, input_grad, weight_grad, parts):
    """Every tile that a size of a type can take, with ragged experts and edges; the plan says that it is taken."""
    print("case", dtype, inf, outf, experts, tokens, flush=True)
    for grad in ("fp32", "bf16") if dtype == "bf16" else ("fp32",):
        c = Case(inf, outf, ragged(experts, tokens), dtype, grad)
        assert launch_shapes(c.plan, tokens, True) == [forward, input_grad, weight_grad, parts]
        c.check_all()
        c = Case(inf, outf, ragged(experts, tokens - 7, 1), dtype, grad, extra=7, pad=(8, 16), seed=1)
        c.check_all()


@pytest.mark.gpu
@pytest.mark.parametrize("other", [torch.float16, torch.int16])
def test_tensors_of_another_type_are_refused(other):
    c = Case(64, 72, [3, 4], "bf16")
    y = torch.empty(7, 72, device=DEV, dtype=torch.bfloat16)
    for bad in (dict(x=c.x.to(other)), dict(w=c.w.to(other)), dict(y=y.to(other))):
        a = dict(x=c.x, w=c.w, y=y) | bad
        with pytest.raises(ValueError, match="bfloat16"):
            B.ar_experts_forward(c.plan, a["x"], a["w"], a["y"], c.ends)
    with pytest.raises(ValueError, match="float32"):
        B.ar_experts_weight_grad(c.plan, c.x, c.dy, torch.empty(c.arena, device=DEV, dtype=torch.int32), c.ends)
    B.ar_experts_destroy(c.plan)


@pytest.mark.gpu
def test_refused_calls_leave_the_plan_unbound():
    """Tensors of another device, or of wrong sizes: the plan can still be bound where it belongs."""
    c = Case(64, 72, [3, 4], "bf16")
    y = c.rows(72, 0, 0)
    for bad in (dict(x=OnDevice(c.x, 1)), dict(w=OnDevice(c.w, 1)), dict(y=y[:5]), dict(ends=OnDevice(c.ends, 1))):
        a = dict(x=c.x, w=c.w, y=y, ends=c.ends) | bad
        with pytest.raises(ValueError):
            B.ar_experts_forward(c.plan, a["x"], a["w"], a["y"], a["ends"])
        assert B.ar_experts_stats(c.plan)["device"] == -1
    B.ar_experts_forward(c.plan, c.x, c.w, y, c.ends)
    torch.cuda.synchronize()
    assert B.ar_experts_stats(c.plan)["device"] == 0
    c.check_rows(y, c.x, False)
    B.ar_experts_destroy(c.plan)


@pytest.mark.gpu
def test_an_unprepared_plan_does_not_end_a_capture_on_another_stream():
    """The call's stream is being captured while another one is current: the call is refused before it allocates,
    and the capture goes on."""
    c = Case(64, 32, [5, 0, 20], "bf16")
    y, other = c.rows(32, 0, 0), torch.zeros(4, device=DEV)
    s, current = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        with torch.cuda.stream(current):
            with pytest.raises((B.ArError, ValueError)):
                B.ar_experts_forward(c.plan, c.x, c.w, y, c.ends, s)
        other.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert other.tolist() == [1] * 4 and B.ar_experts_stats(c.plan)["device"] == -1
    B.ar_experts_destroy(c.plan)
