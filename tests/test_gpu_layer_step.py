"""A training step of an expert layer in 8 bits on two virtual ranks, as its
parts are used together: norm, products, gradients into the arenas, all-reduce,
norm of the gradients, clipping, update, quantisation of the new weights.  Each
part is compared with fp64 on what the parts before it left, with the
tolerances of its own tests; captured and replayed, the step gives the same
bits."""
import math

import pytest
import torch

from gradient_all_reduce_ar_amd import _binding as B
from tests.test_gpu_qexperts import block_tops, blocks, scale_values, spread
from tests.test_gpu_rmsnorm import DEEP, FP8, POW2, U, backward_wanted, check_codes

DEV = "cuda:0"
BF = torch.bfloat16
RANKS, EXPERTS, INF, OUTF, TOKENS = 2, 3, 272, 144, 200
COUNTS = [[90, 0, 107], [20, 150, 30]]  # rows of each rank's experts; some rows are nobody's
MOST, LR = 0.05, 0.02


class Rank:
    def __init__(self, r):
        g = torch.Generator(device=DEV)
        g.manual_seed(r)
        n = lambda *s: torch.randn(s, generator=g, device=DEV)
        self.x, self.residual = n(TOKENS, INF).to(BF), (2 * n(TOKENS, INF)).to(BF)
        self.dy, self.dh = (1e-2 * n(TOKENS, OUTF)).to(BF), (1e-2 * n(TOKENS, INF)).to(BF)
        ends = torch.tensor(COUNTS[r], device=DEV, dtype=torch.int32).cumsum(0, dtype=torch.int32)
        self.ends = ends
        e = lambda *s, dt=BF: torch.zeros(s, device=DEV, dtype=dt)
        self.h, self.y, self.rstd = e(TOKENS, INF), e(TOKENS, INF), e(TOKENS, dt=torch.float32)
        self.codes, self.scales = e(TOKENS, INF, dt=torch.uint8).view(FP8), e(TOKENS, blocks(INF), dt=torch.uint8).view(POW2)
        self.out, self.dxn, self.dx = e(TOKENS, OUTF), e(TOKENS, INF), e(TOKENS, INF)
        self.qdy, self.sdy = e(TOKENS, OUTF, dt=torch.uint8), e(TOKENS, blocks(OUTF), dt=torch.uint8)


class Layer:
    def __init__(self):
        counts = [OUTF * INF] * EXPERTS + [INF]  # the experts' weights and the norm's gain
        self.buckets = B.ar_bucket_plan_create(RANKS, 1, counts, "fp32", "ring", 1 << 18)
        self.offsets, self.size = B.ar_bucket_layout(self.buckets, len(counts))
        self.gain_at = self.offsets[EXPERTS]
        self.held = torch.zeros(self.size, dtype=torch.bool, device=DEV)
        for o, n in zip(self.offsets, counts):
            self.held[o:o + n] = True
        at = self.offsets[:EXPERTS]
        self.norm = B.ar_rmsnorm_create(INF, "bf16", "bf16", "fp32", 1e-5)
        self.wide = B.ar_experts_create(EXPERTS, INF, OUTF, "bf16", "fp32", at)
        self.q = B.ar_qexperts_create(EXPERTS, INF, OUTF, "bf16", at)
        self.clip = B.ar_norm_plan_create(counts, "fp32", self.offsets)
        self.muon = B.ar_muon_plan_create([(OUTF, INF)] * EXPERTS, "fp32", "fp32", at)
        for f, p in ((B.ar_rmsnorm_prepare, self.norm), (B.ar_experts_prepare, self.wide), (B.ar_qexperts_prepare, self.q),
                     (B.ar_norm_plan_prepare, self.clip), (B.ar_muon_plan_prepare, self.muon)):
            f(p)
        g = torch.Generator(device=DEV)
        g.manual_seed(99)
        self.w0 = torch.randn(self.size, generator=g, device=DEV) * 0.05
        self.gain = (1 + 0.1 * torch.randn(INF, generator=g, device=DEV)).to(BF)
        self.ranks = [Rank(r) for r in range(RANKS)]
        self.arenas = [torch.zeros(self.size, device=DEV) for _ in range(RANKS)]
        self.w, self.momentum = self.w0.clone(), torch.zeros(self.size, device=DEV)
        self.codes = torch.full((self.size,), 0x55, device=DEV, dtype=torch.uint8)
        self.scales = torch.zeros(EXPERTS, blocks(OUTF), blocks(INF), device=DEV, dtype=torch.uint8)
        self.clipped, self.total = torch.zeros(self.size, device=DEV), torch.zeros(1, device=DEV)
        self.each = torch.zeros(EXPERTS + 1, device=DEV)
        self.summed = torch.zeros(self.size, device=DEV)

    def start(self):
        self.w.copy_(self.w0)
        self.momentum.zero_()
        B.ar_qexperts_quantize(self.q, self.w, self.codes, self.scales)

    def step(self, s):
        for k, a in zip(self.ranks, self.arenas):
            B.ar_rmsnorm_forward(self.norm, k.x, self.gain, residual=k.residual, h=k.h, y=k.y, codes=k.codes, scales=k.scales,
                                 rstd=k.rstd, stream=s)
            B.ar_qexperts_forward(self.q, k.codes, k.scales, self.codes, self.scales, k.out, k.ends, s)
            B.ar_quantize_rows(k.dy, k.qdy, k.sdy, s)
            B.ar_qexperts_input_grad(self.q, k.qdy, k.sdy, self.codes, self.scales, k.dxn, k.ends, s)
            B.ar_experts_weight_grad(self.wide, k.y, k.dy, a, k.ends, stream=s)
            B.ar_rmsnorm_backward(self.norm, k.dxn, k.h, self.gain, k.rstd, k.dx, a[self.gain_at:self.gain_at + INF], dh=k.dh,
                                  stream=s)
        B.ar_bucket_allreduce(self.buckets, self.arenas, s)
        self.summed.copy_(self.arenas[0])
        B.ar_grad_norm(self.clip, self.arenas[0], self.total, self.each, scale=1 / RANKS, stream=s)
        B.ar_grad_clip(self.clip, self.arenas[0], self.total, MOST, out=self.clipped, stream=s)
        B.ar_muon_step(self.muon, self.clipped, self.momentum, self.w, LR, grad_scale=1 / RANKS, stream=s)
        B.ar_qexperts_quantize(self.q, self.w, self.codes, self.scales, s)

    def state(self):
        out = [self.w, self.momentum, self.codes, self.scales, self.clipped, self.total, self.each, self.summed]
        for k in self.ranks:
            out += [k.h, k.y, k.codes.view(torch.uint8), k.scales.view(torch.uint8), k.out, k.dxn, k.dx]
        return [t.clone() for t in out]

    def destroy(self):
        B.ar_bucket_plan_destroy(self.buckets)
        for f, p in ((B.ar_rmsnorm_destroy, self.norm), (B.ar_experts_destroy, self.wide), (B.ar_qexperts_destroy, self.q),
                     (B.ar_norm_plan_destroy, self.clip), (B.ar_muon_plan_destroy, self.muon)):
            f(p)


@pytest.mark.gpu
def test_step():
    m = Layer()
    m.start()
    codes0, scales0 = m.codes.clone(), m.scales.clone()
    m.step(None)
    torch.cuda.synchronize()
    grads = torch.zeros(m.size, device=DEV, dtype=torch.float64)
    room = torch.zeros_like(grads)
    for r, k in enumerate(m.ranks):
        assert torch.equal(k.h, (k.x.float() + k.residual.float()).to(BF))
        check_codes(k.codes, k.scales, (k.h.float() * k.rstd[:, None]) * m.gain.float())
        check_codes(k.qdy, k.sdy, k.dy)
        lo, n = 0, sum(COUNTS[r])
        assert (k.out[n:] == 0).all() and (k.dxn[n:] == 0).all()
        for e, rows in enumerate(COUNTS[r]):
            s, o = slice(lo, lo + rows), m.offsets[e]
            lo += rows
            if not rows:
                continue
            w = codes0[o:o + OUTF * INF].view(FP8).view(OUTF, INF).double()
            w = w * spread(spread(scale_values(scales0[e]), 0, OUTF), 1, INF)
            for got, q, sc, b in ((k.out, k.codes, k.scales, w.t().contiguous()), (k.dxn, k.qdy, k.sdy, w)):
                a = q[s].view(FP8).double() * spread(scale_values(sc[s].contiguous()), 1, q.shape[1])
                want, mag = a @ b, a.abs() @ b.abs()
                tol = (blocks(q.shape[1]) + 2) * 2.0 ** -23 * mag + 2.0 ** -9 * (block_tops(a) @ block_tops(b.t()).t().contiguous())
                assert ((got[s].double() - want).abs() <= tol + 2.0 ** -8 * (1 + 2.0 ** -7) * want.abs() + 1e-37).all()
            dyt, y = k.dy[s].double().t().contiguous(), k.y[s].double()
            grads[o:o + OUTF * INF] += (dyt @ y).view(-1)
            room[o:o + OUTF * INF] += (rows + 2) * 2.0 ** -23 * (dyt.abs() @ y.abs()).view(-1)
        dx, tol, dg, mag = backward_wanted(k.dxn, k.h, m.gain, k.rstd, k.dh)
        assert ((k.dx.double() - dx).abs() <= tol + 2.0 ** -8 * (1 + 2.0 ** -7) * dx.abs() + 1e-37).all()
        part = slice(m.gain_at, m.gain_at + INF)
        grads[part] += dg
        room[part] += (TOKENS + DEEP) * U * mag
    # two ranks: one more addition
    assert ((m.summed.double() - grads).abs() <= room + 4 * U * grads.abs() + 1e-37)[m.held].all()
    norm = float((m.summed[m.held].double() / RANKS).square().sum().sqrt())
    assert abs(float(m.total) - norm) <= (U + 2.0 ** -30) * norm and norm > MOST
    c = MOST / (norm + 1e-6)
    want = m.summed.double() * c
    assert ((m.clipped.double() - want).abs() <= 4 * U * want.abs() + 1e-37)[m.held].all()
    for e, o in enumerate(m.offsets[:EXPERTS]):
        part = slice(o, o + OUTF * INF)
        assert abs(float(m.each[e]) - float(m.summed[part].double().square().sum().sqrt()) / RANKS) <= 2 * U * norm
        assert ((m.momentum[part].double() - m.clipped[part].double() / RANKS).abs() <= U * m.clipped[part].double().abs()).all()
        moved = (m.w[part] - m.w0[part]).double().view(OUTF, INF)
        # singular values near 1 (0.68 to 1.21) times the step: 144 of them
        assert 0.5 * LR * math.sqrt(OUTF) < float(moved.norm()) < 1.3 * LR * math.sqrt(OUTF)
        rows = m.w[part].view(OUTF, INF)
        value = scale_values(m.scales[e])
        tops = torch.stack([block_tops(p).amax(0) for p in rows.split(128, 0)]).double()
        assert (tops <= 448 * value).all() and (tops > 224 * value).all()
        q = m.codes[part].view(FP8).view(OUTF, INF).double() * spread(spread(value, 0, OUTF), 1, INF)
        # half a step of three fraction bits, or of the smallest codes'
        near = rows.double().abs() * 2.0 ** -4 + spread(spread(value, 0, OUTF), 1, INF) * 2.0 ** -10
        assert ((q - rows.double()).abs() <= near).all()
    m.destroy()


@pytest.mark.gpu
def test_step_captured():
    m = Layer()
    m.start()
    m.step(None)  # (the bucket plan's own tables)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step(torch.cuda.current_stream())
    for _ in range(3):
        for a in m.arenas:
            a.zero_()
        m.start()
        m.step(None)
        m.step(None)
        torch.cuda.synchronize()
        want = m.state()
        for a in m.arenas:
            a.zero_()
        m.start()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(m.state(), want))
    m.destroy()
