"""Cases that measure the grouped expert products and the Muon update.

The operators: the products of a mixture-of-experts layer grouped by expert,
with ragged row counts (forward, input gradient, weight gradient), and the
update of weight matrices by Newton-Schulz orthogonalisation (the
orthogonalisation alone, and the whole Muon step).

``own`` false: plain torch, in fp32.  ``own`` true: the library's calls.
``exact`` is the definition in fp64.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TORCH = {"fp32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "bf16": 2}
NS_COEFFS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
NS_EPS = 1e-7
LR, MU, DECAY = 0.02, 0.95, 0.01


# ------------------------------------------------------------------- cases

def _experts(name, op, tokens, experts, active, inf, outf, dtype="bf16", grad="fp32"):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "active": active, "in": inf, "out": outf,
            "dtype": dtype, "grad": grad}


def _muon(name, op, shapes, grad, weight, ranks):
    return {"name": name, "op": op, "shapes": shapes, "grad": grad, "weight": weight, "ranks": ranks}


def listed():
    return [
        # one decoded token sent to two of eight small experts: latency
        _experts("forward_one_token", "forward", 2, 8, 2, 1024, 512),
        # a decode batch of 16 requests, each to two of 32 experts: every active weight is read once
        _experts("forward_decode_batch", "forward", 32, 32, 20, 4096, 1536),
        # a training batch through the [12288, 4096] gate projection, held by 8 experts
        _experts("forward_gate_proj", "forward", 16384, 8, 8, 4096, 12288),
        # single-precision experts of a small model
        _experts("forward_fp32", "forward", 3001, 8, 7, 1024, 1536, dtype="fp32"),
        # the input gradient of 64 experts, ragged, some of them empty
        _experts("input_grad_batch", "input_grad", 16384, 64, 61, 2048, 1408),
        # sizes that no tile or vector divides
        _experts("input_grad_odd", "input_grad", 777, 5, 4, 1001, 515),
        # weight gradients into an fp32 gradient arena
        _experts("weight_grad_batch", "weight_grad", 16384, 64, 61, 2048, 1408),
        # few rows per expert, bf16 gradients, odd sizes: the arena's writes
        _experts("weight_grad_odd", "weight_grad", 515, 24, 17, 1025, 511, grad="bf16"),
        # four attention-head sized matrices: latency
        _muon("orthogonalize_heads", "orthogonalize", "64x64*4", "bf16", "bf16", 16),
        # a bucket of a small model's matrices, wide, tall, odd, fp32
        _muon("orthogonalize_bucket", "orthogonalize", "1024x1024*4,1024x2048*2,2048x1024*2,515x1001", "fp32", "fp32",
              32),
        # the [12288, 4096] gate-projection gradient in bf16, fp32 weights
        _muon("muon_gate_proj", "muon_step", "12288x4096", "bf16", "fp32", 64),
        # a layer's matrices trained in bf16
        _muon("muon_layer_bf16", "muon_step", "2048x2048*4,5632x2048*2,2048x5632", "bf16", "bf16", 48),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _feature(rng, lo, hi):
    """A feature count: mostly a multiple of 64, now and then odd."""
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.25 else max(lo, n // 64 * 64)


def draw(rng):
    if rng.random() < 0.6:
        op = rng.choice(["forward", "input_grad", "weight_grad"])
        experts = _log_int(rng, 1, 64)
        inf, outf = _feature(rng, 64, 4096), _feature(rng, 64, 4096)
        tokens = _log_int(rng, 1, 16384)
        active = min(experts, tokens, rng.randint(max(1, experts // 2), experts))
        dtype = "fp32" if rng.random() < 0.2 else "bf16"
        grad = "fp32" if dtype == "fp32" else rng.choice(["fp32", "bf16"])
        return _experts(None, op, tokens, experts, active, inf, outf, dtype, grad)
    kinds = []
    budget = 4096.0 ** 3
    for _ in range(rng.randint(1, 6)):
        r, c = _feature(rng, 32, 4096), _feature(rng, 32, 4096)
        if min(r, c) ** 2 * max(r, c) <= budget:
            n = rng.randint(1, 4)
            kinds.append("%dx%d*%d" % (r, c, n))
            budget -= n * min(r, c) ** 2 * max(r, c)
    op = rng.choice(["orthogonalize", "muon_step"])
    grad, weight = rng.choice([("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16")])
    return _muon(None, op, ",".join(kinds) or "64x48", grad, weight, rng.choice([8, 32, 128]))


def _shapes(case):
    out = []
    for part in case["shapes"].split(","):
        size, _, n = part.partition("*")
        r, c = size.split("x")
        out += [(int(r), int(c))] * int(n or 1)
    return out


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _counts(case, seed):
    """Rows of each expert: `active` of them hold at least one, popularity is skewed."""
    rng = np.random.default_rng([int(seed), 5])
    e, a, t = case["experts"], case["active"], case["tokens"]
    who = rng.permutation(e)[:a]
    counts = np.zeros(e, np.int64)
    counts[who] = 1 + rng.multinomial(t - a, rng.dirichlet(np.full(a, 4.0)))
    return counts


def _expert_inputs(case, seed):
    g, dt = _gen(seed), TORCH[case["dtype"]]
    t, e, i, o = case["tokens"], case["experts"], case["in"], case["out"]

    def normal(shape, sigma):
        return torch.randn(shape, generator=g, device=DEV).mul_(sigma).to(dt)

    counts = _counts(case, seed)
    ends = torch.from_numpy(np.cumsum(counts).astype(np.int32)).to(DEV)
    d = {"counts": [int(c) for c in counts], "ends": ends}
    if case["op"] != "input_grad":
        d["x"] = normal((t, i), 1.0)
    if case["op"] != "forward":
        d["dy"] = normal((t, o), 1e-3)
    if case["op"] != "weight_grad":
        d["w"] = normal((e, o, i), 1 / math.sqrt(i))
    return d


def _muon_inputs(case, seed):
    """Gradients of a decaying spectrum (a sum of a few outer products) under
    the noise of a batch, momentum of the same kind, weights; matrices back to
    back."""
    g, shapes, ranks = _gen(seed), _shapes(case), case["ranks"]
    total = sum(r * c for r, c in shapes)

    def arena():
        flat, at = torch.empty(total, device=DEV), 0
        for r, c in shapes:
            k = min(r, c, ranks)
            m = flat[at:at + r * c].view(r, c)
            left = torch.randn((r, k), generator=g, device=DEV)
            left.mul_(torch.logspace(0, -2, k, device=DEV))
            torch.mm(left, torch.randn((k, c), generator=g, device=DEV), out=m)
            m.add_(torch.randn((r, c), generator=g, device=DEV), alpha=0.5).mul_(1e-3)
            at += r * c
        return flat

    d = {"shapes": shapes, "grads": arena().to(TORCH[case["grad"]])}
    if case["op"] == "muon_step":
        d["momentum"] = arena().mul_(5.0)
        d["weights"] = torch.randn(total, generator=g, device=DEV).mul_(0.02).to(TORCH[case["weight"]])
    return d


class _Plan:
    """A plan of the library, destroyed with the state that holds it."""

    def __init__(self, handle, destroy):
        self.handle, self.destroy = handle, destroy

    def __del__(self):
        self.destroy(self.handle)


def prepare(case, seed):
    d = _muon_inputs(case, seed) if "shapes" in case else _expert_inputs(case, seed)
    d["case"] = case
    if not own:
        return d
    from gradient_all_reduce_ar_amd import _binding as ar

    d["ar"] = ar
    if "shapes" in case:
        d["plan"] = _Plan(ar.ar_muon_plan_create(d["shapes"], case["grad"], case["weight"]), ar.ar_muon_plan_destroy)
        ar.ar_muon_plan_prepare(d["plan"].handle)
        d["out"] = torch.empty(d["grads"].numel(), device=DEV, dtype=TORCH[case["weight"]])
        if case["op"] == "muon_step":
            d["momentum_out"] = torch.empty_like(d["momentum"])
        return d
    e, i, o, t = case["experts"], case["in"], case["out"], case["tokens"]
    d["plan"] = _Plan(ar.ar_experts_create(e, i, o, case["dtype"], case["grad"]), ar.ar_experts_destroy)
    ar.ar_experts_prepare(d["plan"].handle)
    if case["op"] == "weight_grad":
        d["out"] = torch.empty((e, o, i), device=DEV, dtype=TORCH[case["grad"]])
    else:
        d["out"] = torch.empty((t, o if case["op"] == "forward" else i), device=DEV, dtype=TORCH[case["dtype"]])
    return d


# --------------------------------------------------------------------- run

def _own(s):
    ar, case, plan = s["ar"], s["case"], s["plan"].handle
    stream = torch.cuda.current_stream()
    if case["op"] == "forward":
        ar.ar_experts_forward(plan, s["x"], s["w"], s["out"], s["ends"], stream)
    elif case["op"] == "input_grad":
        ar.ar_experts_input_grad(plan, s["dy"], s["w"], s["out"], s["ends"], stream)
    elif case["op"] == "weight_grad":
        ar.ar_experts_weight_grad(plan, s["x"], s["dy"], s["out"], s["ends"], stream=stream)
    elif case["op"] == "orthogonalize":
        ar.ar_orthogonalize(plan, s["grads"], s["out"], stream)
    else:
        ar.ar_muon_step(plan, s["grads"], s["momentum"], s["weights"], lr=LR, mu=MU, weight_decay=DECAY,
                        momentum_out=s["momentum_out"], weights_out=s["out"], stream=stream)
        return s["momentum_out"], s["out"]
    return s["out"]


def _plain_experts(s):
    case = s["case"]
    t, e, i, o = case["tokens"], case["experts"], case["in"], case["out"]
    op, at = case["op"], 0
    if op == "weight_grad":
        out = torch.zeros((e, o, i), device=DEV, dtype=TORCH[case["grad"]])
    else:
        out = torch.empty((t, o if op == "forward" else i), device=DEV, dtype=TORCH[case["dtype"]])
    for k, n in enumerate(s["counts"]):
        rows = slice(at, at + n)
        at += n
        if n == 0:
            continue
        if op == "forward":
            out[rows] = torch.mm(s["x"][rows].float(), s["w"][k].float().t()).to(out.dtype)
        elif op == "input_grad":
            out[rows] = torch.mm(s["dy"][rows].float(), s["w"][k].float()).to(out.dtype)
        else:
            out[k] = torch.mm(s["dy"][rows].float().t(), s["x"][rows].float()).to(out.dtype)
    return out


def _plain_orthogonalize(u):
    a, b, c = NS_COEFFS
    tall = u.shape[0] > u.shape[1]
    x = u.t().contiguous() if tall else u
    norm = torch.sum(x.double() * x.double()).sqrt()
    x = (x.double() / (norm + NS_EPS)).float()
    for _ in range(NS_STEPS):
        g = torch.mm(x, x.t())
        x = a * x + torch.mm(b * g + c * torch.mm(g, g), x)
    return x.t() if tall else x


def _plain_muon(s):
    case, at = s["case"], 0
    out = torch.empty(s["grads"].numel(), device=DEV, dtype=TORCH[case["weight"]])
    step = case["op"] == "muon_step"
    mom = torch.empty_like(s["momentum"]) if step else None
    for r, c in s["shapes"]:
        part = slice(at, at + r * c)
        at += r * c
        u = s["grads"][part].view(r, c).float()
        if step:
            m = MU * s["momentum"][part].view(r, c) + u
            mom[part] = m.view(-1)
            u = u + MU * m
        x = _plain_orthogonalize(u)
        if step:
            w = s["weights"][part].view(r, c).float()
            x = (1 - LR * DECAY) * w - (LR * math.sqrt(max(1.0, r / c))) * x
        out[part].view(r, c).copy_(x)
    return (mom, out) if step else out


def run(state):
    if own:
        return _own(state)
    return _plain_muon(state) if "shapes" in state["case"] else _plain_experts(state)


# -------------------------------------------------------------------- work

def work(case):
    if "shapes" in case:
        n = sum(r * c for r, c in _shapes(case))
        nbytes = n * (BYTES[case["grad"]] + BYTES[case["weight"]])
        if case["op"] == "muon_step":
            nbytes += n * (4 + 4 + BYTES[case["weight"]])
        # per step: X X^T and A A are symmetric (half of each), and B X
        flops = 0
        for r, c in _shapes(case):
            m, k = min(r, c), max(r, c)
            flops += NS_STEPS * (m * m * k + m * m * m + 2 * m * m * k)
        return {"bytes": nbytes, "flops": flops}
    t, i, o, b = case["tokens"], case["in"], case["out"], BYTES[case["dtype"]]
    if case["op"] == "weight_grad":
        nbytes = t * (i + o) * b + case["experts"] * i * o * BYTES[case["grad"]]
    else:
        nbytes = t * (i + o) * b + case["active"] * i * o * b
    return {"bytes": nbytes + 4 * case["experts"], "flops": 2 * t * i * o}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    if "shapes" in case:
        return _exact_muon(case, seed)
    s = _expert_inputs(case, seed)
    op, lo, outs = case["op"], 0, []
    for k, n in enumerate(s["counts"]):
        hi = lo + n
        if op == "weight_grad":
            outs.append(s["dy"][lo:hi].double().t().contiguous() @ s["x"][lo:hi].double())
        else:
            rows = s["x" if op == "forward" else "dy"][lo:hi].double()
            w = s["w"][k].double()
            outs.append(rows @ (w.t().contiguous() if op == "forward" else w))
        lo = hi
    return torch.stack(outs) if op == "weight_grad" else torch.cat(outs)


def _exact_muon(case, seed):
    s = _muon_inputs(case, seed)
    a, b, c = NS_COEFFS
    flat, moms, at = [], [], 0
    for rows, cols in s["shapes"]:
        end = at + rows * cols
        u = s["grads"][at:end].double().reshape(rows, cols)
        if case["op"] == "muon_step":
            m = s["momentum"][at:end].double().reshape(rows, cols) * MU + u
            moms.append(m.reshape(-1))
            u = u + m * MU
        x = u / (torch.linalg.vector_norm(u) + NS_EPS)
        for _ in range(NS_STEPS):
            if rows <= cols:
                gram = x @ x.t().contiguous()
                x = a * x + (b * gram) @ x + (c * gram) @ (gram @ x)
            else:
                gram = x.t().contiguous() @ x
                x = a * x + x @ (b * gram) + (x @ gram) @ (c * gram)
        if case["op"] == "muon_step":
            w = s["weights"][at:end].double().reshape(rows, cols)
            x = w * (1 - LR * DECAY) - x * (LR * math.sqrt(max(1.0, rows / cols)))
        flat.append(x.reshape(-1))
        at = end
    return (torch.cat(moms), torch.cat(flat)) if case["op"] == "muon_step" else torch.cat(flat)
