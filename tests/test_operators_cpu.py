"""Refusals, statistics and plan checks of the expert products and the Muon
update on a host without a GPU: every bad call is turned away before any
device work."""
import ctypes
import random

import pytest
import torch

from gradient_all_reduce_ar_amd import _binding as B

A = 1 << 20  # stands for a device address: never read, the calls fail first


@pytest.fixture
def experts():
    p = B.ar_experts_create(4, 64, 32, "bf16", "fp32")
    yield p
    B.ar_experts_destroy(p)


@pytest.fixture
def muon():
    p = B.ar_muon_plan_create([(64, 32), (16, 48)], "bf16", "fp32")
    yield p
    B.ar_muon_plan_destroy(p)


def refused(status, fn, *a, **k):
    with pytest.raises(B.ArError) as e:
        fn(*a, **k)
    assert e.value.status == status, str(e.value)
    return str(e.value)


@pytest.mark.parametrize("args,status", [
    ((0, 64, 64, "bf16", "fp32"), B.AR_ERR_INVALID_ARG),
    ((65537, 64, 64, "bf16", "fp32"), B.AR_ERR_INVALID_ARG),
    ((4, 0, 64, "bf16", "fp32"), B.AR_ERR_INVALID_ARG),
    ((4, 64, 0, "bf16", "fp32"), B.AR_ERR_INVALID_ARG),
    ((4, (1 << 22) + 1, 64, "bf16", "fp32"), B.AR_ERR_INVALID_ARG),
    ((4, 64, 64, "int8_ef", "fp32"), B.AR_ERR_INVALID_ARG),
    ((4, 64, 64, "bf16", "bf16_each"), B.AR_ERR_INVALID_ARG),
    ((4, 64, 64, 17, "fp32"), B.AR_ERR_INVALID_ARG),
    ((4, 64, 64, "fp32", "bf16"), B.AR_ERR_UNSUPPORTED),
    ((2, 4, 4, "bf16", "fp32", [0, 15]), B.AR_ERR_INVALID_ARG),  # overlapping matrices
    ((2, 4, 4, "bf16", "fp32", [0, 1 << 62]), B.AR_ERR_INVALID_ARG),
])
def test_experts_create_refuses(args, status):
    refused(status, B.ar_experts_create, *args)


def test_experts_stats():
    p = B.ar_experts_create(3, 5, 7, "bf16", "fp32", [100, 0, 35])
    s = B.ar_experts_stats(p)
    B.ar_experts_destroy(p)
    assert s == {"nexperts": 3, "device": -1, "in_features": 5, "out_features": 7, "elem_bytes": 2, "grad_bytes": 4,
                 "arena_count": 135, "workspace_bytes": 3 * 8 + 3 * 16 * 64 * 128 * 4}


def test_experts_null_plan():
    for fn in (B.ar_experts_forward, B.ar_experts_input_grad, B.ar_experts_weight_grad):
        refused(B.AR_ERR_INVALID_ARG, fn, None, A, A, A, A)
    refused(B.AR_ERR_INVALID_ARG, B.ar_experts_prepare, None)
    B.ar_experts_destroy(None)


def far(k):
    """Addresses that lie far apart."""
    return A + k * (1 << 30)


@pytest.mark.parametrize("change,word", [
    (dict(x=0), "x is NULL"), (dict(x=far(0) + 1), "aligned"), (dict(y=0), "y is NULL"), (dict(y=far(2) + 1), "aligned"),
    (dict(w=0), "arena is NULL"), (dict(w=far(1) + 1), "arena is not aligned"), (dict(ends=0), "ends is NULL"),
    (dict(ends=far(3) + 2), "ends is not aligned"), (dict(xs=63), "stride"), (dict(ys=31), "stride"),
    (dict(xs=(1 << 22) + 1), "stride"), (dict(y=far(0) + 64), "overlaps"), (dict(y=far(1)), "overlaps"),
    (dict(y=far(3)), "overlaps"), (dict(n=1 << 31), "tokens"),
])
def test_experts_forward_refuses(experts, change, word):
    a = dict(x=far(0), w=far(1), y=far(2), ends=far(3), xs=64, ys=32, n=8) | change
    msg = refused(B.AR_ERR_INVALID_ARG, B.ar_experts_forward, experts, a["x"], a["w"], a["y"], a["ends"],
                  ntokens=a["n"], x_stride=a["xs"], y_stride=a["ys"])
    assert word in msg


@pytest.mark.parametrize("change,word", [
    (dict(x=0), "x is NULL"), (dict(dy=0), "dy is NULL"), (dict(g=0), "arena is NULL"),
    (dict(g=far(2) + 2), "arena is not aligned"), (dict(g=far(0)), "overlaps"), (dict(g=far(1)), "overlaps"),
    (dict(g=far(3)), "overlaps"), (dict(ends=0), "ends is NULL"), (dict(n=0, ends=0), "ends is NULL"),
])
def test_experts_weight_grad_refuses(experts, change, word):
    a = dict(x=far(0), dy=far(1), g=far(2), ends=far(3), n=8) | change
    msg = refused(B.AR_ERR_INVALID_ARG, B.ar_experts_weight_grad, experts, a["x"], a["dy"], a["g"], a["ends"],
                  ntokens=a["n"])
    assert word in msg


def test_experts_rows_end_below_32_bits(experts):
    """Rows rounded up to whole tiles and parts stay inside int32."""
    n = (1 << 31) - 65535
    for call in (lambda: B.ar_experts_forward(experts, far(0), far(1), far(2), far(3), ntokens=n),
                 lambda: B.ar_experts_input_grad(experts, far(0), far(1), far(2), far(3), ntokens=n),
                 lambda: B.ar_experts_weight_grad(experts, far(0), far(1), far(2), far(3), ntokens=n)):
        assert "tokens" in refused(B.AR_ERR_INVALID_ARG, call)


def test_experts_binding_checks_tensors(experts):
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not a device tensor"):
        B.ar_experts_forward(experts, x, A, A, A)
    with pytest.raises(ValueError, match="ntokens"):
        B.ar_experts_forward(experts, A, A, A, A)
    with pytest.raises(ValueError, match="own stride"):
        B.ar_experts_forward(experts, x, A, A, A, x_stride=64)
    with pytest.raises(ValueError, match="weight offsets"):
        B.ar_experts_create(3, 4, 4, "bf16", "fp32", [0, 16])


@pytest.mark.parametrize("args", [
    ([(8, 8)], "int8_ef", "fp32"), ([(8, 8)], "fp32", "bf16_each"), ([(8, 8)], "fp32", 9),
    ([((1 << 20) + 1, 1)], "fp32", "fp32"), ([(1 << 20, 1 << 20)], "fp32", "fp32"),
    ([(4, 4), (4, 4)], "fp32", "fp32", [0, 15]), ([(4, 4)], "fp32", "fp32", [1 << 62]),
])
def test_muon_create_refuses(args):
    refused(B.AR_ERR_INVALID_ARG, B.ar_muon_plan_create, *args)


def test_muon_stats(muon):
    s = B.ar_muon_plan_stats(muon)
    assert (s["nmatrices"], s["device"], s["iterations"], s["arena_count"]) == (2, -1, 5, 64 * 32 + 16 * 48)
    assert (s["grad_bytes"], s["weight_bytes"]) == (2, 4)
    assert s["workspace_bytes"] > 0 and s["launches"] > 0
    empty = B.ar_muon_plan_create([(0, 5), (3, 0)], "fp32", "fp32")
    s = B.ar_muon_plan_stats(empty)
    assert s["arena_count"] == 0 and s["workspace_bytes"] == 0 and s["launches"] == 0
    B.ar_muon_plan_destroy(empty)


@pytest.mark.parametrize("n,abc", [
    (0, None), (33, None), (1, [(float("nan"), 0, 0)]), (1, [(float("inf"), 0, 0)]), (1, [(2000.0, 0, 0)]),
    (1, [(0, 0, 1e5)]), (8, [(8.0, 0, 0)] * 8),
])
def test_muon_iterations_refused(muon, n, abc):
    refused(B.AR_ERR_INVALID_ARG, B.ar_muon_plan_set_iterations, muon, n, abc)
    assert B.ar_muon_plan_stats(muon)["iterations"] == 5


def test_muon_iterations_set(muon):
    B.ar_muon_plan_set_iterations(muon, 8, [(1.5, -0.5, 0.0)] * 8)
    assert B.ar_muon_plan_stats(muon)["iterations"] == 8
    B.ar_muon_plan_set_iterations(muon, 3)
    assert B.ar_muon_plan_stats(muon)["iterations"] == 3
    with pytest.raises(ValueError):
        B.ar_muon_plan_set_iterations(muon, 2, [(1, 0, 0)])


def test_muon_scales(muon):
    B.ar_muon_plan_set_scales(muon, [0.5, 2.0])
    B.ar_muon_plan_set_scales(muon)
    refused(B.AR_ERR_INVALID_ARG, B.ar_muon_plan_set_scales, muon, [0.5, float("nan")])
    refused(B.AR_ERR_INVALID_ARG, B.ar_muon_plan_set_scales, muon, [1e40, 1.0])
    with pytest.raises(ValueError):
        B.ar_muon_plan_set_scales(muon, [1.0])


def test_muon_null_plan():
    refused(B.AR_ERR_INVALID_ARG, B.ar_orthogonalize, None, A, A)
    refused(B.AR_ERR_INVALID_ARG, B.ar_muon_step, None, A, A, A, lr=0.1)
    refused(B.AR_ERR_INVALID_ARG, B.ar_muon_plan_prepare, None)
    refused(B.AR_ERR_INVALID_ARG, B.ar_muon_plan_set_iterations, None, 5)
    refused(B.AR_ERR_INVALID_ARG, B.ar_muon_plan_set_scales, None)
    B.ar_muon_plan_destroy(None)


@pytest.mark.parametrize("g,o,word", [
    (0, far(1), "grads is NULL"), (far(0), 0, "out is NULL"), (far(0) + 1, far(1), "aligned"),
    (far(0), far(1) + 2, "aligned"), (far(0), far(0) + 64, "overlap"), (far(0), far(0), "overlap"),  # bf16 and fp32
])
def test_orthogonalize_refuses(muon, g, o, word):
    assert word in refused(B.AR_ERR_INVALID_ARG, B.ar_orthogonalize, muon, g, o)


@pytest.mark.parametrize("change,word", [
    (dict(g=0), "grads is NULL"), (dict(m=0), "momentum is NULL"), (dict(w=0), "NULL"),
    (dict(m=far(1) + 2), "aligned"), (dict(m=far(0)), "overlap"), (dict(w=far(0)), "overlap"),
    (dict(w=far(1)), "overlap"), (dict(mo=far(2)), "overlap"), (dict(wo=far(1)), "overlap"),
    (dict(wo=far(2) + 64), "overlap"), (dict(mo=far(1) + 64), "overlap"), (dict(lr=float("nan")), "finite"),
    (dict(mu=float("inf")), "finite"), (dict(decay=1e40, lr=1.0), "finite"), (dict(gs=1e39), "finite"),
])
def test_muon_step_refuses(muon, change, word):
    a = dict(g=far(0), m=far(1), w=far(2), mo=None, wo=None, lr=0.1, mu=0.9, decay=0.0, gs=1.0) | change
    msg = refused(B.AR_ERR_INVALID_ARG, B.ar_muon_step, muon, a["g"], a["m"], a["w"], a["lr"], mu=a["mu"],
                  weight_decay=a["decay"], grad_scale=a["gs"], momentum_out=a["mo"], weights_out=a["wo"])
    assert word in msg


def test_muon_params_null(muon):
    L = B.lib()
    assert L.ar_muon_step(muon, far(0), far(1), far(2), None, None, None, None) == B.AR_ERR_INVALID_ARG
    assert b"params" in L.ar_last_error()


def test_muon_offsets_from_a_bucket_plan():
    """The tensor offsets of a bucket layout are valid matrix and weight offsets."""
    shapes = [(16, 32), (7, 5), (64, 64)]
    bp = B.ar_bucket_plan_create(2, 1, [r * c for r, c in shapes], "bf16", "ring", 4096)
    offs, arena = B.ar_bucket_layout(bp, len(shapes))
    B.ar_bucket_plan_destroy(bp)
    p = B.ar_muon_plan_create(shapes, "bf16", "bf16", offs)
    assert B.ar_muon_plan_stats(p)["arena_count"] <= arena
    B.ar_muon_plan_destroy(p)


def test_c_struct_sizes():
    """The ctypes mirrors have the C layout."""
    assert ctypes.sizeof(B.ar_experts_stats_t) == 56
    assert ctypes.sizeof(B.ar_muon_stats_t) == 48
    assert ctypes.sizeof(B.ar_muon_params_t) == 40


# ------------------------------------------------------ Muon work lists

SPLIT, WHOLE = True, False
# matrices, and per product (X X^T, b A + c A A + a I, B X) the tile and whether tiles are cut; what the GPU tests
# of the tiled kernels run
TILED = {
    "small": ([(160, 224), (300, 200), (131, 517), (5, 3)], [(64, WHOLE), (64, WHOLE), (64, WHOLE)]),
    "wide": ([(1000, 4100)], [(64, WHOLE), (64, WHOLE), (128, WHOLE)]),
    "tall": ([(2100, 1990)], [(256, SPLIT), (128, WHOLE), (128, WHOLE)]),
    "equal": ([(1024, 2048)] * 8, [(128, WHOLE), (128, WHOLE), (256, WHOLE)]),
    "large": ([(2050, 2060)] * 2 + [(2061, 2049)] * 2, [(256, WHOLE), (256, WHOLE), (256, SPLIT)]),
    "square": ([(4001, 4100)], [(256, SPLIT), (256, SPLIT), (256, SPLIT)]),
    "long": ([(300, 5000)] * 3 + [(5001, 299)] * 3, [(256, SPLIT), (64, WHOLE), (256, WHOLE)]),
    "mixed": ([(4000, 520), (520, 4000), (1001, 1003), (64, 64), (2049, 2047)],
              [(256, SPLIT), (128, WHOLE), (128, WHOLE)]),
}


def check_work(shapes, plan):
    """Every tile of every matrix (the upper triangle's of the square products) is covered exactly once along its
    contraction; whole tiles have no partial tile, the pieces of the others have consecutive ones of their own."""
    seen = []
    for product in range(3):
        w = B.ar_muon_plan_work(plan, product)
        side, tiles, slots = w["tile"], {}, []
        assert (w["group"][1:] >= w["group"][:-1]).all() and (w["k1"] > w["k0"]).all()
        for mat, r, c, k0, k1, slot in zip(*(w[k].tolist() for k in ("matrix", "row", "col", "k0", "k1", "slot"))):
            tiles.setdefault((mat, r, c), []).append((slot, k0, k1))
        want = set()
        for i, (rows, cols) in enumerate(shapes):
            m, n = (-(-v // 64) * 64 for v in sorted((rows, cols)))
            if m == 0:
                continue
            up, across = -(-m // side), -(-(m if product < 2 else n) // side)
            mine = {(i, r, c) for r in range(up) for c in range(r if product < 2 else 0, across)}
            want |= mine
            for t in mine:
                pieces = sorted(tiles[t])
                ranges = sorted((k0, k1) for _, k0, k1 in pieces)
                assert ranges[0][0] == 0 and ranges[-1][1] == (n if product == 0 else m)
                assert all(a[1] == b[0] for a, b in zip(ranges, ranges[1:]))
                assert all(k0 % 64 == 0 and k1 % 64 == 0 for k0, k1 in ranges)
                s = [p[0] for p in pieces]
                assert s == [-1] if len(s) == 1 else s == list(range(s[0], s[0] + len(s))) and s[0] >= 0
                slots += s if len(s) > 1 else []
        assert set(tiles) == want
        assert sorted(slots) == list(range(len(slots)))
        seen.append((side, len(slots) > 0))
    return seen


@pytest.mark.parametrize("name", TILED)
@pytest.mark.parametrize("types", [("bf16", "fp32"), ("bf16", "bf16")])
def test_muon_work_lists(name, types):
    shapes, want = TILED[name]
    p = B.ar_muon_plan_create(shapes, *types)
    assert check_work(shapes, p) == want
    s = B.ar_muon_plan_stats(p)
    assert s["launches"] == 2 + 5 * (3 + sum(split for _, split in want))
    B.ar_muon_plan_destroy(p)


@pytest.mark.parametrize("seed", range(12))
def test_muon_work_lists_of_drawn_matrices(seed):
    rng = random.Random(seed)
    shapes = [(int(2 ** rng.uniform(0, 12.5)), int(2 ** rng.uniform(0, 12.5))) for _ in range(rng.randint(1, 9))]
    shapes += [(0, 7), (257, 300)]
    p = B.ar_muon_plan_create(shapes, "fp32", "fp32")
    check_work(shapes, p)
    B.ar_muon_plan_destroy(p)


def test_muon_work_of_small_plans_and_refusals(muon):
    for product in range(3):
        w = B.ar_muon_plan_work(muon, product)
        assert w["tile"] == 0 and len(w["group"]) == 0
    refused(B.AR_ERR_INVALID_ARG, B.ar_muon_plan_work, muon, 3)
    refused(B.AR_ERR_INVALID_ARG, B.ar_muon_plan_work, muon, -1)
    refused(B.AR_ERR_INVALID_ARG, B.ar_muon_plan_work, None, 0)


# ------------------------------------------- which tiles a product takes

# in, out, experts, rows, type: the tile of forward, input gradient and weight gradient, and its parts; what the GPU
# tests of the products' kernels run.  The features of a type's second half are on no vector boundary.
DISPATCH = {
    "bf16": [
        (4104, 1032, 8, 1500, (64, 128), (256, 256), (128, 128), 1),
        (1000, 1200, 40, 4100, (256, 256), (64, 128), (128, 128), 1),
        (520, 264, 1, 6000, (128, 128), (128, 128), (64, 128), 16),
        (2048, 1408, 40, 40, (64, 128), (64, 128), (128, 128), 1),
        (136, 72, 1, 8200, (32, 64), (64, 128), (64, 128), 16),
        (520, 264, 40, 2500, (32, 64), (128, 128), (128, 128), 1),
        (2056, 1000, 8, 2500, (128, 128), (64, 128), (256, 256), 1),
        (521, 263, 1, 6000, (128, 128), (128, 128), (64, 128), 16),
        (2047, 1409, 40, 40, (64, 128), (64, 128), (64, 128), 1),
        (135, 71, 1, 8200, (32, 64), (64, 128), (64, 128), 16),
        (521, 263, 40, 2500, (32, 64), (128, 128), (64, 128), 1),
        (1025, 1001, 8, 2500, (128, 128), (128, 128), (128, 128), 1),
        (2049, 2047, 3, 4000, (64, 128), (64, 128), (128, 128), 1),
    ],
    "fp32": [
        (1000, 1200, 8, 2500, (128, 128), (32, 64), (64, 128), 1),
        (1000, 1200, 1, 1500, (64, 128), (32, 64), (64, 128), 3),
        (520, 264, 40, 6000, (32, 64), (64, 128), (64, 128), 1),
        (136, 72, 1, 8200, (32, 64), (128, 128), (64, 128), 16),
        (1001, 1201, 8, 2500, (128, 128), (32, 64), (64, 128), 1),
        (1001, 1201, 1, 1500, (64, 128), (32, 64), (64, 128), 3),
        (521, 263, 40, 6000, (32, 64), (64, 128), (64, 128), 1),
        (135, 71, 1, 8200, (32, 64), (128, 128), (64, 128), 16),
    ],
}
ROWS_OF_DISPATCH = [(dtype, *row) for dtype in DISPATCH for row in DISPATCH[dtype]]


def launch_shapes(plan, tokens, aligned):
    s = [B.ar_experts_launch_shape(plan, p, tokens, aligned) for p in ("forward", "input_grad", "weight_grad")]
    return [(v["tile_rows"], v["tile_cols"]) for v in s] + [s[2]["parts"]]


@pytest.mark.parametrize("dtype,inf,outf,experts,tokens,forward,input_grad,weight_grad,parts", ROWS_OF_DISPATCH)
def test_experts_launch_shapes(dtype, inf, outf, experts, tokens, forward, input_grad, weight_grad, parts):
    p = B.ar_experts_create(experts, inf, outf, dtype, "fp32")
    assert launch_shapes(p, tokens, True) == [forward, input_grad, weight_grad, parts]
    B.ar_experts_destroy(p)


def test_every_kernel_of_the_products_is_run():
    """The tests' sizes take every tile of every type, with and without whole vectors, that any size takes."""
    def taken(dtype, inf, outf, experts, tokens, aligned):
        p = B.ar_experts_create(experts, inf, outf, dtype, "fp32")
        shapes = launch_shapes(p, tokens, aligned)
        B.ar_experts_destroy(p)
        vec = 8 if dtype == "bf16" else 4
        shapes[2] += (shapes.pop() > 1,)
        return {(dtype, aligned and inf % vec == 0 and outf % vec == 0, k, s) for k, s in enumerate(shapes)}

    few = [("bf16", 64, 64, 4, 4), ("fp32", 64, 64, 4, 4), ("bf16", 71, 135, 4, 4), ("fp32", 71, 135, 4, 4),
           ("bf16", 64, 64, 1, 40), ("fp32", 64, 64, 1, 40), ("bf16", 71, 135, 1, 40), ("fp32", 71, 135, 1, 40)]
    run = set().union(*(taken(*r[:5], True) for r in ROWS_OF_DISPATCH + few))
    rng = random.Random(7)
    for _ in range(1500):
        inf, outf, tokens = (int(2 ** rng.uniform(0, top)) for top in (13, 13, 15))
        if rng.random() < 0.7:
            inf, outf = max(8, inf // 8 * 8), max(8, outf // 8 * 8)
        any_size = taken(rng.choice(["bf16", "fp32"]), inf, outf, int(2 ** rng.uniform(0, 8)), tokens, rng.random() < 0.7)
        assert any_size <= run, any_size - run


def test_experts_launch_shape_refusals_and_nothing(experts):
    assert B.ar_experts_launch_shape(experts, "forward", 0) == dict(tile_rows=0, tile_cols=0, parts=0)
    assert B.ar_experts_launch_shape(experts, "weight_grad", 0)["parts"] == 1
    refused(B.AR_ERR_INVALID_ARG, B.ar_experts_launch_shape, experts, 3, 8)
    refused(B.AR_ERR_INVALID_ARG, B.ar_experts_launch_shape, experts, -1, 8)
    refused(B.AR_ERR_INVALID_ARG, B.ar_experts_launch_shape, None, 0, 8)
    refused(B.AR_ERR_INVALID_ARG, B.ar_experts_launch_shape, experts, 0, 1 << 31)


# --------------------------------------------------- tensors of a call

class OnDevice:
    """A CPU tensor that says that it lies on a device: for checks that come before anything is launched."""

    def __init__(self, t, device=0):
        self.t, self.device, self.is_cuda = t, device, True

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.device


@pytest.fixture
def one_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for stats in ("_experts_info", "_muon_info"):
        monkeypatch.setattr(B, stats, {})


OTHER_TYPES = {"bf16": [torch.float16, torch.int16, torch.uint16, torch.float32], "fp32": [torch.int32, torch.bfloat16, torch.float64]}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_experts_refuse_tensors_of_another_type(dtype, one_device):
    """The type itself is checked: 16 bits may be fp16, 32 bits an integer."""
    p = B.ar_experts_create(2, 8, 16, dtype, "fp32")
    B._experts_of(p).device = 0
    mine = torch.bfloat16 if dtype == "bf16" else torch.float32

    def tensors(**types):
        shapes = dict(x=(6, 8), dy=(6, 16), y=(6, 16), dx=(6, 8), w=(256,), g=(256,))
        return {k: OnDevice(torch.zeros(s, dtype=types.get(k, torch.float32 if k == "g" else mine)))
                for k, s in shapes.items()}

    ends = OnDevice(torch.tensor([2, 6], dtype=torch.int32))
    for other in OTHER_TYPES[dtype]:
        for k in ("x", "w", "y"):
            t = tensors(**{k: other})
            with pytest.raises(ValueError, match="bfloat16|float32"):
                B.ar_experts_forward(p, t["x"], t["w"], t["y"], ends)
        for k in ("dy", "w", "dx"):
            t = tensors(**{k: other})
            with pytest.raises(ValueError, match="bfloat16|float32"):
                B.ar_experts_input_grad(p, t["dy"], t["w"], t["dx"], ends)
        for k in ("x", "dy"):
            t = tensors(**{k: other})
            with pytest.raises(ValueError, match="bfloat16|float32"):
                B.ar_experts_weight_grad(p, t["x"], t["dy"], t["g"], ends)
    for other in OTHER_TYPES["fp32"]:
        t = tensors(g=other)
        with pytest.raises(ValueError, match="float32"):
            B.ar_experts_weight_grad(p, t["x"], t["dy"], t["g"], ends)
    B.ar_experts_destroy(p)


@pytest.mark.parametrize("grad,weight", [("bf16", "fp32"), ("fp32", "bf16")])
def test_muon_refuses_tensors_of_another_type(grad, weight, one_device):
    p = B.ar_muon_plan_create([(4, 8)], grad, weight)
    B._muon_of(p).device = 0
    mine = dict(g=grad, m="fp32", w=weight, mo="fp32", wo=weight)
    name = {"bf16": torch.bfloat16, "fp32": torch.float32}
    for k, own in mine.items():
        for other in OTHER_TYPES[own]:
            t = {n: OnDevice(torch.zeros(32, dtype=other if n == k else name[d])) for n, d in mine.items()}
            with pytest.raises(ValueError, match="bfloat16|float32"):
                B.ar_muon_step(p, t["g"], t["m"], t["w"], 0.1, momentum_out=t["mo"], weights_out=t["wo"])
            if k in ("g", "w"):
                with pytest.raises(ValueError, match="bfloat16|float32"):
                    B.ar_orthogonalize(p, t["g"], t["w"])
    B.ar_muon_plan_destroy(p)


def test_refused_calls_do_not_bind_a_plan(one_device):
    """A call whose tensors lie on another device than the current one, or do not fit, leaves the plan unbound."""
    ex, mu = B.ar_experts_create(2, 8, 16, "fp32"), B.ar_muon_plan_create([(4, 8)], "fp32", "fp32")
    ends = OnDevice(torch.tensor([2, 6], dtype=torch.int32))
    for device, rows in ((1, 6), (0, 5)):
        x, y, w, g = (OnDevice(torch.zeros(s), device) for s in ((6, 8), (rows, 16), (256,), (31 if rows < 6 else 32,)))
        with pytest.raises(ValueError, match="device 1" if device else "wanted"):
            B.ar_experts_forward(ex, x, w, y, ends)
        with pytest.raises(ValueError, match="device 1" if device else "wanted"):
            B.ar_orthogonalize(mu, g, g)
    assert B.ar_experts_stats(ex)["device"] == -1 and B.ar_muon_plan_stats(mu)["device"] == -1
    B.ar_experts_destroy(ex)
    B.ar_muon_plan_destroy(mu)
