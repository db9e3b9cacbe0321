"""The RMS norm, its backward pass and the 8-bit rows against plain fp64
implementations, on cuda:0.

Tolerances.  h is one fp32 addition rounded to the rows' type: compared bit for
bit.  rstd is formed in fp64 and rounded once (2^-24, and 2^-30 for the rest).
y: rstd's rounding, two fp32 products and the rounding to the rows' type.
Codes and scales are a function of the fp32 product h rstd gain, which torch
forms with the same two roundings: compared as numbers, without tolerance.

Backward.  A sum of terms in fp32, each at most DEEP additions deep (8 per
lane's piece of up to 8, six over a wave, up to 16 waves), is off by DEEP 2^-24
of its magnitudes; each elementary operation by 2^-24 of its result.
"""
import pytest
import torch

from gradient_all_reduce_ar_amd import _binding as B

DEV = "cuda:0"
T = {"fp32": torch.float32, "bf16": torch.bfloat16}
FP8, POW2 = torch.float8_e4m3fn, torch.float8_e8m0fnu
U = 2.0 ** -24
DEEP = 64 + 6 + 16 + 4


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rows(t, n, dtype, pad=0, shift=0, seed=0, sigma=1.0, fill=None):
    """[t, n] with a row stride of n + pad, `shift` elements into its storage."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    flat = torch.randn(t * (n + pad) + shift, generator=g, device=DEV).mul_(sigma)
    if fill is not None:
        flat.fill_(fill)
    return flat.to(dtype)[shift:].view(t, n + pad)[:, :n]


def byte_rows(t, n, pad=0, shift=0, like=torch.uint8):
    return torch.full((t * (n + pad) + shift,), 0x55, device=DEV, dtype=torch.uint8)[shift:].view(like).view(t, n + pad)[:, :n]


def quantized(x):
    """The definition, from fp32 or bf16 numbers: code values and scale bytes, in fp64."""
    t, n = x.shape
    b = -(-n // 128)
    v = torch.zeros(t, b * 128, dtype=torch.float64, device=DEV)
    v[:, :n] = x.double()
    v = v.view(t, b, 128)
    top = v.abs().amax(2)
    e = torch.full_like(top, -127)
    for k in range(-127, 121):
        e = torch.where(top > 448 * 2.0 ** k, torch.full_like(e, k + 1), e)
    u = v / torch.exp2(e)[:, :, None]
    _, k = torch.frexp(u)
    step = torch.exp2((k - 1).clamp_min(-6).double() - 3)
    q = torch.round(u / step) * step
    bad = ~torch.isfinite(v).all(2)
    q[bad] = float("nan")
    bytes_ = (e + 127).to(torch.int32)
    bytes_[bad] = 255
    return q.view(t, b * 128)[:, :n], bytes_


def check_codes(codes, scales, x):
    q, s = quantized(x)
    assert torch.equal(scales.view(torch.uint8).to(torch.int32), s), "scales"
    got = codes.view(FP8).double()
    assert torch.equal(got.nan_to_num(1e9), q.nan_to_num(1e9)), f"{int((got != q).sum())} codes"


SHAPES = [(1, 1), (1, 4096), (3, 7), (2, 8), (5, 127), (5, 128), (5, 129), (33, 512), (9, 513), (4, 1000), (17, 1001),
          (1, 2047), (70, 2048), (3, 4099), (2, 8192), (2, 8193), (1, 16384), (3, 20000), (2, 65536), (1, 65535)]
MANY = [(1500, 64), (1100, 1000), (1024, 2048), (1030, 4096), (1025, 5001), (1027, 8200), (1024, 16385), (1024, 40000)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,gain", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("t,n", SHAPES + MANY)
def test_forward(t, n, dtype, gain):
    print("case", t, n, dtype, gain, flush=True)
    dt = T[dtype]
    odd = (t + n) % 2  # dense aligned rows, or rows off every alignment
    pad, shift = (3, 1) if odd else (0, 0)
    x, r = rows(t, n, dt, pad, shift, 1), rows(t, n, dt, pad, shift, 2, 3.0)
    g = rows(1, n, T[gain], 0, shift, 3)[0]
    h, y = rows(t, n, dt, pad, shift, fill=7.0), rows(t, n, dt, pad, shift, fill=7.0)
    b = -(-n // 128)
    codes, scales = byte_rows(t, n, pad, shift, FP8), byte_rows(t, b, pad, shift)
    rstd = torch.zeros(t, device=DEV)
    plan = B.ar_rmsnorm_create(n, dtype, gain, eps=1e-5)
    B.ar_rmsnorm_forward(plan, x, g, residual=r, h=h, y=y, codes=codes, scales=scales, rstd=rstd)
    torch.cuda.synchronize()
    assert torch.equal(h, (x.float() + r.float()).to(dt))
    want = (h.double().square().mean(1) + 1e-5).rsqrt()
    assert ((rstd.double() - want).abs() <= (U + 2.0 ** -30) * want).all()
    full = h.double() * want[:, None] * g.double()
    assert ((y.double() - full).abs() <= (3 * U + half(dt)) * (1 + 2.0 ** -7) * full.abs() + 1e-37).all()
    check_codes(codes, scales, (h.float() * rstd[:, None]) * g.float())
    # without the residual, only some of the outputs, and what lies between the rows
    y2 = rows(t, n, dt, pad, shift, fill=7.0)
    B.ar_rmsnorm_forward(plan, h, g, y=y2)
    codes2, scales2 = byte_rows(t, n, 2, 0), byte_rows(t, b, 0, 0, POW2)
    B.ar_rmsnorm_forward(plan, h, g, codes=codes2, scales=scales2)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(codes.view(torch.uint8), codes2) and torch.equal(scales, scales2.view(torch.uint8))
    for o, w in ((h, n), (y, n), (codes.view(torch.uint8), n), (scales, b)):
        if pad:
            whole = o.as_strided((t - 1, pad), (o.stride(0), 1), o.storage_offset() + w) if t > 1 else o[:0]
            assert (whole.double() == (7.0 if o.dtype != torch.uint8 else 0x55)).all(), "between the rows"
    B.ar_rmsnorm_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("t,n", [(5, 300), (1200, 4096), (3, 40000)])
def test_forward_in_place(t, n, dtype):
    dt = T[dtype]
    x, r, g = rows(t, n, dt, seed=1), rows(t, n, dt, seed=2), rows(1, n, dt, seed=3)[0]
    plan = B.ar_rmsnorm_create(n, dtype)
    h, y = torch.empty_like(x), torch.empty_like(x)
    B.ar_rmsnorm_forward(plan, x, g, residual=r, h=h, y=y)
    a, b = x.clone(), r.clone()
    B.ar_rmsnorm_forward(plan, a, g, residual=b, h=b, y=a)  # the usual pair: the stream and the rows
    torch.cuda.synchronize()
    assert torch.equal(a, y) and torch.equal(b, h)
    a, b = x.clone(), r.clone()
    B.ar_rmsnorm_forward(plan, a, g, residual=b, h=a, y=b)
    torch.cuda.synchronize()
    assert torch.equal(a, h) and torch.equal(b, y)
    B.ar_rmsnorm_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward_of_any_size(dtype):
    """Rows of zeros, far below and above 1, with infinities and NaN: each row is its own."""
    dt, n = T[dtype], 300
    x = rows(9, n, dt, seed=4)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e30
    x[4, 5] = float("inf")
    x[5, 299] = float("nan")
    x[6] *= 1e-40
    x[7, :128] = 0
    g = rows(1, n, dt, seed=5)[0]
    with pytest.raises(B.ArError):  # an rstd that fp32 does not hold
        B.ar_rmsnorm_create(n, dtype, eps=0.0)
    for eps in (1e-6, 1e-75):
        plan = B.ar_rmsnorm_create(n, dtype, eps=eps)
        y, codes, scales, rstd = torch.empty_like(x), byte_rows(9, n), byte_rows(9, 3), torch.zeros(9, device=DEV)
        B.ar_rmsnorm_forward(plan, x, g, y=y, codes=codes, scales=scales, rstd=rstd)
        torch.cuda.synchronize()
        d = x.double()
        want = 1 / (d.square().mean(1) + eps).sqrt()
        assert torch.equal(rstd.isnan(), want.isnan())
        assert ((rstd.double() - want).abs() <= (U + 2.0 ** -30) * want + 2.0 ** -149)[torch.isfinite(want.float())].all()
        assert torch.equal(torch.isinf(rstd), torch.isinf(want.float()))
        exact32 = (x.float() * rstd[:, None]) * g.float()
        assert torch.equal(y.nan_to_num(1e9), exact32.to(dt).nan_to_num(1e9)) and torch.equal(y.isnan(), exact32.isnan())
        check_codes(codes, scales, exact32)
        assert torch.isfinite(y[[0, 2, 3, 6, 7, 8]]).all()
        B.ar_rmsnorm_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("t,n", [(1, 1), (1, 128), (3, 129), (5, 1000), (200, 1408), (1000, 2048), (7, 4099), (4097, 64), (2, 100000)])
def test_quantize_rows(t, n, dtype):
    print("case", t, n, dtype, flush=True)
    odd = (t + n) % 2
    pad, shift = (5, 1) if odd else (0, 0)
    x = rows(t, n, T[dtype], pad, shift, 1) * torch.exp2(torch.randint(-60, 60, (t, 1), device=DEV).float()).to(T[dtype])
    x = rows(t, n, T[dtype], pad, shift, fill=0.0).copy_(x)
    b = -(-n // 128)
    codes, scales = byte_rows(t, n, pad, shift), byte_rows(t, b, pad, shift)
    B.ar_quantize_rows(x, codes, scales)
    torch.cuda.synchronize()
    check_codes(codes, scales, x)
    if pad and t > 1:
        for o, w in ((codes, n), (scales, b)):
            assert (o.as_strided((t - 1, pad), (o.stride(0), 1), o.storage_offset() + w) == 0x55).all()


@pytest.mark.gpu
def test_quantize_borders():
    """Largest magnitudes on both sides of 448 2^e, ties, the smallest and largest numbers, zeros, infinities, NaN."""
    tops = [448.0, 448.0 * (1 + 2.0 ** -23), 448.0 * (1 - 2.0 ** -24), 1.0, 1.75, 1.7500001, 2.0 ** -126, 448 * 2.0 ** -127, 3e-38,
            2.0 ** -149, 1e-44, 0.0, 3.4e38, 448 * 2.0 ** 118, 464.0, float("inf"), float("nan"), -448.0, -1e-10, -0.0]
    x = torch.zeros(len(tops), 256, device=DEV)
    steps = torch.arange(127, device=DEV) / 127.0
    for i, v in enumerate(tops):
        x[i, 0] = v
        if abs(v) < 1e39:
            x[i, 1:128] = steps * v * 0.999
            x[i, 128:] = torch.arange(128, device=DEV) * 0.0625 * 2.0 ** (i - 10)  # many ties
    codes, scales = byte_rows(len(tops), 256), byte_rows(len(tops), 2)
    B.ar_quantize_rows(x, codes, scales)
    torch.cuda.synchronize()
    check_codes(codes, scales, x)
    assert (codes[15, :128] == 0x7f).all() and int(scales[15, 0]) == 255 and (scales[:, 1] != 255).all()


def backward_wanted(dy, h, g, rstd, dh):
    dy, h, g, r = dy.double(), h.double(), g.double(), rstd.double()[:, None]
    xhat, u = h * r, dy * g
    terms = u * xhat
    mean = terms.mean(1, keepdim=True)
    dx = r * (u - xhat * mean)
    tol = r * (DEEP * U * terms.abs().mean(1, keepdim=True) * xhat.abs() + 6 * U * (u.abs() + (xhat * mean).abs()))
    if dh is not None:
        tol = tol + U * (dx.abs() + dh.double().abs())
        dx = dx + dh.double()
    each = dy * xhat
    return dx, tol, each.sum(0), each.abs().sum(0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,gain,grad", [("bf16", "bf16", "fp32"), ("bf16", "fp32", "bf16"), ("fp32", "fp32", "fp32")])
@pytest.mark.parametrize("t,n", SHAPES + MANY + [(5000, 7), (3001, 1001), (2600, 513)])
def test_backward(t, n, dtype, gain, grad):
    print("case", t, n, dtype, gain, grad, flush=True)
    dt = T[dtype]
    odd = (t + n) % 2
    pad, shift = (3, 1) if odd else (0, 0)
    dy, h, dh = (rows(t, n, dt, pad, shift, k, s) for k, s in ((1, 1e-3), (2, 2.0), (3, 1e-3)))
    g = rows(1, n, T[gain], 0, shift, 4)[0]
    rstd = (h.double().square().mean(1) + 1e-6).rsqrt().float()
    plan = B.ar_rmsnorm_create(n, dtype, gain, grad)
    for residual, accumulate in ((True, False), (False, True)):
        dx = rows(t, n, dt, pad, shift, fill=7.0)
        dg = torch.full((n + shift,), 0.5, device=DEV, dtype=T[grad])[shift:]
        B.ar_rmsnorm_backward(plan, dy, h, g, rstd, dx, dg, dh=dh if residual else None, accumulate=accumulate)
        torch.cuda.synchronize()
        want, tol, wg, mag = backward_wanted(dy, h, g, rstd, dh if residual else None)
        off = (dx.double() - want).abs()
        assert (off <= tol + half(dt) * (1 + 2.0 ** -7) * want.abs() + 1e-37).all(), float((off / tol).max())
        if accumulate:
            wg, mag = wg + 0.5, mag + 0.5
        depth = min(t, 64 + t // 64) + 100
        assert ((dg.double() - wg).abs() <= depth * U * mag + half(T[grad]) * (1 + 2.0 ** -7) * wg.abs() + 1e-37).all()
        if pad and t > 1:
            assert (dx.as_strided((t - 1, pad), (dx.stride(0), 1), dx.storage_offset() + n) == 7).all()
    B.ar_rmsnorm_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["dy", "h", "dh"])
@pytest.mark.parametrize("dtype,t,n", [("bf16", 1300, 2048), ("fp32", 37, 1001), ("bf16", 3, 40000)])
def test_backward_in_place(which, dtype, t, n):
    dt = T[dtype]
    d = {k: rows(t, n, dt, seed=i) for i, k in enumerate(("dy", "h", "dh"))}
    g = rows(1, n, dt, seed=7)[0]
    rstd = (d["h"].double().square().mean(1) + 1e-6).rsqrt().float()
    plan = B.ar_rmsnorm_create(n, dtype)
    dx, dg, dg2 = torch.empty_like(d["h"]), torch.empty_like(g), torch.empty_like(g)
    B.ar_rmsnorm_backward(plan, d["dy"], d["h"], g, rstd, dx, dg, dh=d["dh"])
    B.ar_rmsnorm_backward(plan, d["dy"], d["h"], g, rstd, d[which], dg2, dh=d["dh"])
    torch.cuda.synchronize()
    assert torch.equal(d[which], dx) and torch.equal(dg, dg2)
    B.ar_rmsnorm_destroy(plan)


@pytest.mark.gpu
def test_backward_no_rows():
    plan = B.ar_rmsnorm_create(300, "bf16", "fp32", "fp32")
    e, g = torch.empty(0, 300, device=DEV, dtype=torch.bfloat16), torch.ones(300, device=DEV)
    dg, r = torch.full((300,), 3.0, device=DEV), torch.empty(0, device=DEV)
    B.ar_rmsnorm_backward(plan, e, e, g, r, e, dg, accumulate=True)
    torch.cuda.synchronize()
    assert (dg == 3).all()
    B.ar_rmsnorm_backward(plan, e, e, g, r, e, dg)
    B.ar_rmsnorm_forward(plan, e, g, y=e)
    torch.cuda.synchronize()
    assert (dg == 0).all()
    B.ar_rmsnorm_destroy(plan)


@pytest.mark.gpu
def test_backward_against_differences():
    """dx and dgain against central differences, in fp64, of the forward definition."""
    t, n, eps = 3, 21, 1e-3
    x, g, w = rows(t, n, torch.float32, seed=1), rows(1, n, torch.float32, seed=2)[0], rows(t, n, torch.float32, seed=3)

    def loss(x, g):  # the gradient of y is w, of h 0.25
        r = 1 / (x.square().mean(1, keepdim=True) + eps).sqrt()
        return float((x * r * g * w.double()).sum() + 0.25 * x.sum())

    plan = B.ar_rmsnorm_create(n, "fp32", eps=eps)
    y, rstd, dx, dg = torch.empty_like(x), torch.empty(t, device=DEV), torch.empty_like(x), torch.empty_like(g)
    B.ar_rmsnorm_forward(plan, x, g, y=y, rstd=rstd)
    B.ar_rmsnorm_backward(plan, w, x, g, rstd, dx, dg, dh=torch.full_like(x, 0.25))
    torch.cuda.synchronize()
    step = 1e-4  # truncation: step^2 times third derivatives of order 10; rounding: 1e-15 / step
    for i in range(t):
        for j in range(n):
            d = torch.zeros(t, n, device=DEV, dtype=torch.float64)
            d[i, j] = step
            want = (loss(x.double() + d, g.double()) - loss(x.double() - d, g.double())) / (2 * step)
            assert abs(float(dx[i, j]) - want) <= 1e-5
    for j in range(n):
        d = torch.zeros(n, device=DEV, dtype=torch.float64)
        d[j] = step
        want = (loss(x.double(), g.double() + d) - loss(x.double(), g.double() - d)) / (2 * step)
        assert abs(float(dg[j]) - want) <= 1e-5
    B.ar_rmsnorm_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("t,n", [(2000, 1000), (600, 4096)])
def test_captured_and_streams(t, n):
    """Forward and backward in a graph, replayed on changing rows with eager calls between; forward calls of one
    plan on two streams; the same bits every time."""
    x, r = rows(t, n, torch.bfloat16, seed=1), rows(t, n, torch.bfloat16, seed=2)
    g = rows(1, n, torch.bfloat16, seed=3)[0]
    plan = B.ar_rmsnorm_create(n, "bf16", "bf16", "fp32")
    b = -(-n // 128)

    def outputs():
        return {"h": torch.zeros_like(x), "y": torch.zeros_like(x), "codes": byte_rows(t, n), "scales": byte_rows(t, b),
                "rstd": torch.zeros(t, device=DEV)}

    def step(o, dx, dg, s):
        B.ar_rmsnorm_forward(plan, x, g, residual=r, stream=s, **o)
        B.ar_rmsnorm_backward(plan, o["y"], o["h"], g, o["rstd"], dx, dg, dh=r, stream=s)

    one, two = outputs(), outputs()
    dx, dg, dx2, dg2 = torch.zeros_like(x), torch.zeros(n, device=DEV), torch.zeros_like(x), torch.zeros(n, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(ValueError, match="prepared"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            step(one, dx, dg, torch.cuda.current_stream())
    B.ar_rmsnorm_prepare(plan)
    with torch.cuda.graph(graph):
        step(one, dx, dg, torch.cuda.current_stream())
    for k in range(4):
        x.copy_(rows(t, n, torch.bfloat16, seed=10 + k))
        graph.replay()
        torch.cuda.synchronize()
        step(two, dx2, dg2, None)
        torch.cuda.synchronize()
        assert all(torch.equal(one[k], two[k]) for k in one) and torch.equal(dx, dx2) and torch.equal(dg, dg2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [outputs() for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for o, s in zip(outs, streams):
            B.ar_rmsnorm_forward(plan, x, g, residual=r, stream=s, **o)
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], two[k]) for o in outs for k in o)
    B.ar_rmsnorm_destroy(plan)


@pytest.mark.gpu
def test_far_rows():
    """Elements past 2^31: the last rows of a long batch, with a stride that is not theirs."""
    t, n, stride = 33000, 64, 65537
    flat = torch.zeros(t * stride, device=DEV, dtype=torch.bfloat16)
    x = flat.view(t, stride)[:, :n]
    x.copy_(rows(t, n, torch.bfloat16, seed=1))
    g = torch.ones(n, device=DEV, dtype=torch.bfloat16)
    plan = B.ar_rmsnorm_create(n, "bf16")
    y, codes, scales = torch.empty(t, n, device=DEV, dtype=torch.bfloat16), byte_rows(t, n), byte_rows(t, 1)
    B.ar_rmsnorm_forward(plan, x, g, y=y)
    B.ar_quantize_rows(x, codes, scales)
    torch.cuda.synchronize()
    part = slice(t - 100, t)
    d = x[part].double()
    full = d * (d.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    assert ((y[part].double() - full).abs() <= (3 * U + 2.0 ** -8) * full.abs() + 1e-37).all()
    check_codes(codes[part], scales[part], x[part])
    B.ar_rmsnorm_destroy(plan)


@pytest.mark.gpu
def test_tensor_checks():
    plan = B.ar_rmsnorm_create(64, "bf16")
    x, g = rows(4, 64, torch.bfloat16), rows(1, 64, torch.bfloat16)[0]
    y = torch.empty_like(x)
    for bad, word in ((x.float(), "wanted"), (x[:, :32], "wanted"), (x.cpu(), "device tensor"), (x.t().contiguous().t(), "contiguous")):
        with pytest.raises(ValueError, match=word):
            B.ar_rmsnorm_forward(plan, bad, g, y=y)
    for kw in (dict(y=y[:3]), dict(y=y, rstd=torch.empty(3, device=DEV)), dict(codes=byte_rows(4, 64).view(torch.int8), scales=byte_rows(4, 1)),
               dict(codes=byte_rows(4, 64), scales=byte_rows(4, 2)), dict(y=y, residual=x.float())):
        with pytest.raises(ValueError):
            B.ar_rmsnorm_forward(plan, x, g, **kw)
    with pytest.raises(ValueError, match="wanted"):
        B.ar_quantize_rows(x.half(), byte_rows(4, 64), byte_rows(4, 1))
    with pytest.raises(ValueError, match="wanted"):
        B.ar_quantize_rows(x, byte_rows(4, 63), byte_rows(4, 1))
    B.ar_rmsnorm_destroy(plan)


@pytest.mark.gpu
def test_forward_needs_no_workspace():
    """A program that only runs forward, eager and captured, never pays for the backward pass's workspace."""
    t, n = 70, 1000
    x, g = rows(t, n, torch.bfloat16, seed=1), rows(1, n, torch.bfloat16, seed=2)[0]
    y, z = torch.zeros_like(x), torch.zeros_like(x)
    plan = B.ar_rmsnorm_create(n, "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.ar_rmsnorm_forward(plan, x, g, y=y, stream=torch.cuda.current_stream())
    assert B.ar_rmsnorm_stats(plan)["device"] == -1
    for k in range(3):
        x.copy_(rows(t, n, torch.bfloat16, seed=3 + k))
        graph.replay()
        B.ar_rmsnorm_forward(plan, x, g, y=z)
        torch.cuda.synchronize()
        assert torch.equal(y, z) and float(y.abs().max()) > 0
    assert B.ar_rmsnorm_stats(plan)["device"] == -1
    r, dx, dg = torch.ones(t, device=DEV), torch.empty_like(x), torch.empty_like(g)
    with pytest.raises(ValueError, match="prepared"):  # the backward pass has one
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            B.ar_rmsnorm_backward(plan, x, x, g, r, dx, dg, stream=torch.cuda.current_stream())
    B.ar_rmsnorm_backward(plan, x, x, g, r, dx, dg)
    assert B.ar_rmsnorm_stats(plan)["device"] == 0
    B.ar_rmsnorm_forward(plan, x, g, y=y)
    torch.cuda.synchronize()
    assert torch.equal(y, z)
    B.ar_rmsnorm_destroy(plan)
