"""Cases that measure gradient clipping, the RMS norm and the 8-bit expert products.

The operators: the global norm of a gradient arena and its clipping; the root-
mean-square norm with the residual's addition and an output in 8 bits (forward,
and the backward pass); the products of a mixture-of-experts layer in 8-bit
floating point with a scale, a power of two, for each block of 128 (forward,
input gradient with the quantisation of its rows, quantisation of the weights).

``own`` false: plain torch, in fp32 and fp64.  ``own`` true: the library's
calls.  ``exact`` is the definition in fp64.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TORCH = {"fp32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "bf16": 2}
FP8, POW2 = torch.float8_e4m3fn, torch.float8_e8m0fnu  # codes, and scales: 2^(byte - 127)
BLOCK, TOP = 128, 448.0      # elements of a scale block; the largest e4m3 number
EPS = 1e-6                   # of the RMS norm
CLIP_EPS = 1e-6


# ------------------------------------------------------------------- cases

def _clip(name, tensors, median, spread, dtype, max_norm):
    return {"name": name, "op": "clip", "tensors": tensors, "median": median, "spread": spread, "dtype": dtype,
            "max_norm": max_norm}


def _norm(name, op, tokens, features, dtype, gain, residual, y, codes):
    return {"name": name, "op": op, "tokens": tokens, "features": features, "dtype": dtype, "gain": gain,
            "residual": residual, "y": y, "codes": codes}


def _product(name, op, tokens, experts, active, inf, outf, dtype="bf16"):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "active": active, "in": inf, "out": outf,
            "dtype": dtype}


def listed():
    return [
        # the gradients of four attention-head sized matrices: latency
        _clip("clip_heads", 4, 4096, 0.0, "bf16", 0.05),
        # the bucketed bf16 gradients of 300 tensors, from 512 bytes to 64 MiB, at any element's address
        _clip("clip_bucketed", 300, 131072, 2.0, "bf16", 1.0),
        # one decoded token: the residual and the 8-bit input of the next product
        _norm("norm_one_token", "norm", 1, 4096, "bf16", "bf16", True, False, True),
        # a training batch: the residual, the 16-bit rows for the weight gradient, the 8-bit ones for the product
        _norm("norm_batch", "norm", 16384, 4096, "bf16", "bf16", True, True, True),
        # the backward pass of that batch, the gradient of the residual path added
        _norm("norm_grad_batch", "norm_grad", 16384, 4096, "bf16", "bf16", True, False, False),
        # single-precision rows that no vector divides
        _norm("norm_grad_odd", "norm_grad", 3001, 1001, "fp32", "fp32", False, False, False),
        # one decoded token sent to two of eight small experts: latency
        _product("forward_one_token", "forward", 2, 8, 2, 1024, 512),
        # a decode batch of 16 requests, each to two of 32 experts: every active weight is read once
        _product("forward_decode_batch", "forward", 32, 32, 20, 4096, 1536),
        # a training batch through the [12288, 4096] gate projection, held by 8 experts
        _product("forward_gate_proj", "forward", 16384, 8, 8, 4096, 12288),
        # the input gradient of 64 experts, ragged, some of them empty, from 16-bit rows
        _product("input_grad_batch", "input_grad", 16384, 64, 61, 2048, 1408),
        # sizes that no tile, block or vector divides, fp32 results
        _product("input_grad_odd", "input_grad", 777, 5, 4, 1001, 515, dtype="fp32"),
        # the fp32 weights of 64 experts after an update
        _product("quantize_experts", "quantize", 1, 64, 1, 2048, 1408, dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _feature(rng, lo, hi):
    """A feature count: mostly a multiple of 64, now and then odd."""
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.25 else max(lo, n // 64 * 64)


def draw(rng):
    kind = rng.random()
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind < 0.25:
        tensors = _log_int(rng, 1, 2000)
        median = _log_int(rng, 64, min(1 << 24, (1 << 26) // tensors))
        return _clip(None, tensors, median, round(rng.uniform(0.0, 1.5), 3), dtype, round(10 ** rng.uniform(-2, 1), 4))
    if kind < 0.55:
        features = _feature(rng, 64, 8192)
        tokens = _log_int(rng, 1, min(32768, (1 << 26) // features))
        gain = "fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"])
        if rng.random() < 0.5:
            return _norm(None, "norm_grad", tokens, features, dtype, gain, rng.random() < 0.7, False, False)
        y, codes = rng.choice([(True, False), (False, True), (True, True)])
        return _norm(None, "norm", tokens, features, dtype, gain, rng.random() < 0.7, y, codes)
    experts = _log_int(rng, 1, 64)
    inf, outf = _feature(rng, 64, 4096), _feature(rng, 64, 4096)
    op = rng.choice(["forward", "forward", "input_grad", "input_grad", "quantize"])
    tokens = 1 if op == "quantize" else _log_int(rng, 1, 16384)
    active = min(experts, tokens, rng.randint(max(1, experts // 2), experts))
    return _product(None, op, tokens, experts, active, inf, outf, dtype)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _layout(case):
    """Element counts and offsets of the tensors, and the arena's length: tensors back to back in buckets of about
    25 MiB, each of which starts on 256 bytes (of the sizes alone, as a model's are)."""
    rng = np.random.default_rng([case["tensors"], case["median"]])
    size = BYTES[case["dtype"]]
    counts = np.round(rng.lognormal(math.log(case["median"]), case["spread"], case["tensors"]))
    counts = np.clip(counts, 1, (64 << 20) // size).astype(np.int64)
    offsets, at, start, align = [], 0, 0, 256 // size
    for n in counts:
        if at > start and (at + int(n) - start) * size > 25 << 20:
            at = start = -(-at // align) * align
        offsets.append(at)
        at += int(n)
    return [int(n) for n in counts], offsets, at


def _clip_inputs(case, seed):
    g = _gen(seed)
    counts, offsets, total = _layout(case)
    held = torch.zeros(total, dtype=torch.int32, device=DEV)
    ends = torch.tensor([o + n for o, n in zip(offsets, counts) if o + n < total], device=DEV, dtype=torch.int64)
    held[torch.tensor(offsets, device=DEV)] += 1
    held[ends] -= 1
    held = held.cumsum(0, dtype=torch.int32).to(torch.bool)
    grads = torch.randn(total, generator=g, device=DEV).mul_(1e-3).to(TORCH[case["dtype"]])
    return {"counts": counts, "offsets": offsets, "held": held, "grads": grads}


def _rows(g, shape, sigma, dt):
    """Activations: a few features are far larger than the others."""
    x = torch.randn(shape, generator=g, device=DEV)
    loud = torch.rand(shape[-1], generator=g, device=DEV) < 0.004
    return x.mul_(sigma * (1 + 19 * loud.float())).to(dt)


def _norm_inputs(case, seed):
    g, dt = _gen(seed), TORCH[case["dtype"]]
    shape = (case["tokens"], case["features"])
    d = {"gain": torch.randn(shape[1], generator=g, device=DEV).mul_(0.1).add_(1).to(TORCH[case["gain"]])}
    if case["op"] == "norm":
        d["x"] = _rows(g, shape, 0.5, dt)
        if case["residual"]:
            d["residual"] = _rows(g, shape, 1.0, dt)
        return d
    d["h"] = _rows(g, shape, 1.0, dt)
    d["dy"] = torch.randn(shape, generator=g, device=DEV).mul_(1e-3).to(dt)
    if case["residual"]:
        d["dh"] = torch.randn(shape, generator=g, device=DEV).mul_(1e-3).to(dt)
    d["rstd"] = (d["h"].double().square().mean(1) + EPS).rsqrt().float()  # what the forward pass left
    return d


def _scale_bytes(top):
    """Biased exponents of the least powers of two (2^-127 at least) with top <= 448 2^e."""
    m, k = torch.frexp(top)
    return (k + 118 + (m > 0.875)).clamp_min(0)


def _quantized(v, scale_bytes):
    """e4m3 codes of v 2^-e (which is exact)."""
    return (v * ((254 - scale_bytes).to(torch.int32) << 23).view(torch.float32)).to(FP8)


def _quantized_rows(x):
    """Codes [rows, features] and scales [rows, blocks] of fp32 rows."""
    t, n = x.shape
    blocks = -(-n // BLOCK)
    v = torch.nn.functional.pad(x, (0, blocks * BLOCK - n)).view(t, blocks, BLOCK)
    e = _scale_bytes(v.abs().amax(2))
    codes = _quantized(v, e[:, :, None]).view(t, blocks * BLOCK)[:, :n].contiguous()
    return codes, e.to(torch.uint8).view(POW2)


def _quantized_weights(w):
    """Codes [experts, out, in] and scales [experts, out blocks, in blocks] of fp32 matrices."""
    e, o, i = w.shape
    ob, ib = -(-o // BLOCK), -(-i // BLOCK)
    v = torch.nn.functional.pad(w, (0, ib * BLOCK - i, 0, ob * BLOCK - o)).view(e, ob, BLOCK, ib, BLOCK)
    p = _scale_bytes(v.abs().amax((2, 4)))
    codes = _quantized(v, p[:, :, None, :, None]).view(e, ob * BLOCK, ib * BLOCK)[:, :o, :i].contiguous()
    return codes, p.to(torch.uint8).contiguous().view(POW2)


def _counts(case, seed):
    """Rows of each expert: `active` of them hold at least one, popularity is skewed."""
    rng = np.random.default_rng([int(seed), 5])
    e, a, t = case["experts"], case["active"], case["tokens"]
    who = rng.permutation(e)[:a]
    counts = np.zeros(e, np.int64)
    counts[who] = 1 + rng.multinomial(t - a, rng.dirichlet(np.full(a, 4.0)))
    return counts


def _product_inputs(case, seed):
    g, dt = _gen(seed), TORCH[case["dtype"]]
    t, e, i, o = case["tokens"], case["experts"], case["in"], case["out"]
    w = torch.randn((e, o, i), generator=g, device=DEV).mul_(1 / math.sqrt(i))
    if case["op"] == "quantize":
        return {"w": w.to(dt)}
    counts = _counts(case, seed)
    d = {"counts": [int(c) for c in counts], "ends": torch.from_numpy(np.cumsum(counts).astype(np.int32)).to(DEV)}
    d["w"], d["w_scales"] = _quantized_weights(w)
    if case["op"] == "forward":
        d["x"], d["x_scales"] = _quantized_rows(_rows(g, (t, i), 1.0, torch.float32))
    else:
        d["dy"] = torch.randn((t, o), generator=g, device=DEV).mul_(1e-3).to(dt)
    return d


def _inputs(case, seed):
    if case["op"] == "clip":
        return _clip_inputs(case, seed)
    return _norm_inputs(case, seed) if "features" in case else _product_inputs(case, seed)


class _Plan:
    """A plan of the library, destroyed with the state that holds it."""

    def __init__(self, handle, destroy):
        self.handle, self.destroy = handle, destroy

    def __del__(self):
        self.destroy(self.handle)


def _new(shape, dtype):
    return torch.zeros(shape, device=DEV, dtype=dtype)


def prepare(case, seed):
    d = _inputs(case, seed)
    d["case"], op, dt = case, case["op"], TORCH[case["dtype"]]
    # the program's buffers
    if op == "clip":
        d["out"], d["norm"] = torch.zeros_like(d["grads"]), _new(1, torch.float32)
    elif "features" in case:
        t, n = case["tokens"], case["features"]
        if op == "norm":
            d["h"] = _new((t, n), dt) if case["residual"] else None
            d["y"] = _new((t, n), dt) if case["y"] else None
            d["rstd"] = _new(t, torch.float32) if case["y"] else None  # a training step keeps it
            d["codes"] = _new((t, n), torch.uint8).view(FP8) if case["codes"] else None
            d["scales"] = _new((t, -(-n // BLOCK)), torch.uint8).view(POW2) if case["codes"] else None
        else:
            d["dx"], d["dgain"] = _new((t, n), dt), _new(n, torch.float32)
    else:
        t, e, i, o = case["tokens"], case["experts"], case["in"], case["out"]
        if op == "forward":
            d["out"] = _new((t, o), dt)
        elif op == "input_grad":
            d["out"] = _new((t, i), dt)
            d["codes"] = _new((t, o), torch.uint8).view(FP8)
            d["scales"] = _new((t, -(-o // BLOCK)), torch.uint8).view(POW2)
        else:
            d["codes"] = _new((e, o, i), torch.uint8).view(FP8)
            d["scales"] = _new((e, -(-o // BLOCK), -(-i // BLOCK)), torch.uint8).view(POW2)
    if own:
        from gradient_all_reduce_ar_amd import _binding as ar

        d["ar"] = ar
        if op == "clip":
            d["plan"] = _Plan(ar.ar_norm_plan_create(d["counts"], case["dtype"], d["offsets"]), ar.ar_norm_plan_destroy)
            ar.ar_norm_plan_prepare(d["plan"].handle)
        elif "features" in case:
            d["plan"] = _Plan(ar.ar_rmsnorm_create(case["features"], case["dtype"], case["gain"], "fp32", EPS),
                              ar.ar_rmsnorm_destroy)
            ar.ar_rmsnorm_prepare(d["plan"].handle)
        else:
            d["plan"] = _Plan(ar.ar_qexperts_create(case["experts"], case["in"], case["out"], case["dtype"]),
                              ar.ar_qexperts_destroy)
            ar.ar_qexperts_prepare(d["plan"].handle)
    return d


# --------------------------------------------------------------------- run

def _own(s):
    ar, case, plan = s["ar"], s["case"], s["plan"].handle
    stream, op = torch.cuda.current_stream(), case["op"]
    if op == "clip":
        ar.ar_grad_norm(plan, s["grads"], s["norm"], stream=stream)
        ar.ar_grad_clip(plan, s["grads"], s["norm"], case["max_norm"], out=s["out"], stream=stream)
        return s["norm"], s["out"]
    if op == "norm":
        ar.ar_rmsnorm_forward(plan, s["x"], s["gain"], residual=s.get("residual"), h=s["h"], y=s["y"], codes=s["codes"],
                              scales=s["scales"], rstd=s["rstd"], stream=stream)
        return s["h"], s["y"], s["rstd"], s["codes"], s["scales"]
    if op == "norm_grad":
        ar.ar_rmsnorm_backward(plan, s["dy"], s["h"], s["gain"], s["rstd"], s["dx"], s["dgain"], dh=s.get("dh"),
                               stream=stream)
        return s["dx"], s["dgain"]
    if op == "forward":
        ar.ar_qexperts_forward(plan, s["x"], s["x_scales"], s["w"], s["w_scales"], s["out"], s["ends"], stream)
        return s["out"]
    if op == "input_grad":
        ar.ar_quantize_rows(s["dy"], s["codes"], s["scales"], stream)
        ar.ar_qexperts_input_grad(plan, s["codes"], s["scales"], s["w"], s["w_scales"], s["out"], s["ends"], stream)
        return s["out"], s["codes"], s["scales"]
    ar.ar_qexperts_quantize(plan, s["w"], s["codes"], s["scales"], stream)
    return s["codes"], s["scales"]


def _plain_clip(s):
    case = s["case"]
    g = torch.where(s["held"], s["grads"], 0).float()
    norm = (g.double() * g.double()).sum().sqrt().float()
    c = (case["max_norm"] / (norm.double() + CLIP_EPS)).clamp_max(1.0).float()
    return norm.view(1), (g * c).to(s["grads"].dtype)


def _plain_norm(s):
    case, dt = s["case"], TORCH[s["case"]["dtype"]]
    h = s["x"]
    if case["residual"]:
        h = (h.float() + s["residual"].float()).to(dt)
    f = h.float()
    rstd = 1 / ((f.double() * f.double()).mean(1) + EPS).sqrt()
    y = f * rstd.float()[:, None] * s["gain"].float()
    codes, scales = _quantized_rows(y) if case["codes"] else (None, None)
    return (h if case["residual"] else None, y.to(dt) if case["y"] else None, rstd.float() if case["y"] else None,
            codes, scales)


def _plain_norm_grad(s):
    case, dt = s["case"], TORCH[s["case"]["dtype"]]
    dy = s["dy"].float()
    xhat = s["h"].float() * s["rstd"][:, None]
    u = dy * s["gain"].float()
    mean = (u * xhat).mean(1, keepdim=True, dtype=torch.float64).float()
    dx = (u - xhat * mean) * s["rstd"][:, None]
    if case["residual"]:
        dx = dx + s["dh"].float()
    return dx.to(dt), (dy * xhat).sum(0, dtype=torch.float64).float()


def _wide_rows(codes, scales):
    return codes.float() * scales.float().repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _wide_weight(codes, scales):
    s = scales.float().repeat_interleave(BLOCK, 0)[:codes.shape[0]].repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]
    return codes.float() * s


def _plain_product(s):
    case = s["case"]
    if case["op"] == "quantize":
        return _quantized_weights(s["w"].float())
    forward, at, dt = case["op"] == "forward", 0, TORCH[case["dtype"]]
    codes, scales = (s["x"], s["x_scales"]) if forward else _quantized_rows(s["dy"].float())
    rows = _wide_rows(codes, scales)
    out = torch.empty((case["tokens"], case["out" if forward else "in"]), device=DEV, dtype=dt)
    for k, n in enumerate(s["counts"]):  # (the groups are ragged)
        if n == 0:
            continue
        w = _wide_weight(s["w"][k], s["w_scales"][k])
        out[at:at + n] = torch.mm(rows[at:at + n], w.t() if forward else w).to(dt)
        at += n
    return out if forward else (out, codes, scales)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "clip":
        return _plain_clip(state)
    if op == "norm":
        return _plain_norm(state)
    return _plain_norm_grad(state) if op == "norm_grad" else _plain_product(state)


# -------------------------------------------------------------------- work

def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "clip":
        n = sum(_layout(case)[0])
        return {"bytes": 2 * n * b, "flops": 3 * n}
    if "features" in case:
        n, t, gain = case["tokens"] * case["features"], case["tokens"], case["features"] * BYTES[case["gain"]]
        blocks = t * -(-case["features"] // BLOCK)
        if case["op"] == "norm":
            nbytes = n * b * (1 + 2 * case["residual"] + case["y"]) + (n + blocks) * case["codes"] + 4 * t * case["y"]
            return {"bytes": nbytes + gain, "flops": 6 * n}
        return {"bytes": n * b * (3 + case["residual"]) + 4 * t + gain + 4 * case["features"], "flops": 10 * n}
    t, e, i, o = case["tokens"], case["experts"], case["in"], case["out"]
    blocks = -(-o // BLOCK) * -(-i // BLOCK)
    if case["op"] == "quantize":
        return {"bytes": e * (i * o * (b + 1) + blocks), "flops": 3 * e * i * o}
    k, n = (i, o) if case["op"] == "forward" else (o, i)
    rows = t * (k + -(-k // BLOCK))
    if case["op"] == "input_grad":
        rows += t * k * b  # the quantised rows are an output
    return {"bytes": rows + t * n * b + case["active"] * (i * o + blocks) + 4 * e, "flops": 2 * t * i * o}


# ------------------------------------------------------------------- exact

def _spread_scales(s, dim, n):
    """Each scale as often as its block has elements, along `dim`."""
    at = torch.arange(n, device=DEV) // BLOCK
    return s.index_select(dim, at)


def _exact_scales(top):
    """The least powers of two, 2^-127 at least, whose 448-fold is no less than top."""
    e = torch.ceil(torch.log2((top / TOP).clamp_min(2.0 ** -140)))
    e = torch.where(top > TOP * torch.exp2(e), e + 1, e)  # where the logarithm was rounded
    e = torch.where(top <= TOP * torch.exp2(e - 1), e - 1, e)
    return torch.exp2(e.clamp_min(-127))


def _exact_codes(v, scales):
    """e4m3 codes, as numbers, of v / scales: rounded to a multiple of 2^(exponent - 3), of 2^-9 at least."""
    u = v / scales
    _, e = torch.frexp(u)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return torch.round(u / step) * step


def _exact_rows(x):
    blocks = torch.split(x.abs(), BLOCK, dim=1)
    scales = _exact_scales(torch.stack([b.amax(1) for b in blocks], 1))
    return _exact_codes(x, _spread_scales(scales, 1, x.shape[1])), scales


def _exact_clip(case, seed):
    s = _clip_inputs(case, seed)
    g = s["grads"].double()
    out, total = torch.zeros_like(g), torch.zeros((), device=DEV, dtype=torch.float64)
    for o, n in zip(s["offsets"], s["counts"]):
        total += g[o:o + n].square().sum()
    norm = total.sqrt()
    c = min(1.0, case["max_norm"] / (float(norm) + CLIP_EPS))
    for o, n in zip(s["offsets"], s["counts"]):
        out[o:o + n] = g[o:o + n] * c
    return norm.view(1), out


def _exact_norm(case, seed):
    s = _norm_inputs(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if case["residual"]:
            h = (h + s["residual"].double()).to(TORCH[case["dtype"]]).double()  # the norm is that of the stored sum
        rstd = (h.square().sum(1) / h.shape[1] + EPS).pow(-0.5)
        y = h * rstd.view(-1, 1) * s["gain"].double().view(1, -1)
        codes, scales = _exact_rows(y) if case["codes"] else (None, None)
        return (h if case["residual"] else None, y if case["y"] else None, rstd if case["y"] else None, codes, scales)
    h, dy, gain, r = s["h"].double(), s["dy"].double(), s["gain"].double(), s["rstd"].double().view(-1, 1)
    dx = r * gain * dy - h * r ** 3 * (h * gain * dy).sum(1, keepdim=True) / h.shape[1]
    if case["residual"]:
        dx = dx + s["dh"].double()
    return dx, (dy * h * r).sum(0)


def _exact_product(case, seed):
    s = _product_inputs(case, seed)
    op, lo, outs = case["op"], 0, []
    if op == "quantize":
        codes, scales = [], []
        for w in s["w"]:
            w = w.double()
            top = torch.stack([torch.stack([p.amax() for p in r.split(BLOCK, 1)]) for r in w.abs().split(BLOCK, 0)])
            scales.append(_exact_scales(top))
            wide = _spread_scales(_spread_scales(scales[-1], 0, w.shape[0]), 1, w.shape[1])
            codes.append(_exact_codes(w, wide))
        return torch.stack(codes), torch.stack(scales)
    codes, scales = (s["x"].double(), s["x_scales"].double()) if op == "forward" else _exact_rows(s["dy"].double())
    rows = codes * _spread_scales(scales, 1, codes.shape[1])
    for k, n in enumerate(s["counts"]):
        w, ws = s["w"][k].double(), s["w_scales"][k].double()
        w = w * _spread_scales(_spread_scales(ws, 0, w.shape[0]), 1, w.shape[1])
        outs.append(rows[lo:lo + n].contiguous() @ (w.t().contiguous() if op == "forward" else w))
        lo += n
    out = torch.cat(outs)
    return out if op == "forward" else (out, codes, scales)


def exact(case, seed):
    if case["op"] == "clip":
        return _exact_clip(case, seed)
    return _exact_norm(case, seed) if "features" in case else _exact_product(case, seed)
