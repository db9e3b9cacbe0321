"""Refusals, statistics and plan checks of gradient clipping, the RMS norm and
the 8-bit rows and expert products on a host without a GPU: every bad call is
turned away before any device work."""
import ctypes

import pytest
import torch

from gradient_all_reduce_ar_amd import _binding as B
from tests.test_operators_cpu import far, refused

BAD = B.AR_ERR_INVALID_ARG


@pytest.fixture
def norm():
    p = B.ar_norm_plan_create([10, 0, 500], "bf16", [3, 7, 100])
    yield p
    B.ar_norm_plan_destroy(p)


@pytest.fixture
def rms():
    p = B.ar_rmsnorm_create(300, "bf16", "fp32", "fp32")
    yield p
    B.ar_rmsnorm_destroy(p)


@pytest.fixture
def experts():
    p = B.ar_qexperts_create(4, 300, 200, "bf16")
    yield p
    B.ar_qexperts_destroy(p)


# ------------------------------------------------------ norm and clipping

@pytest.mark.parametrize("args", [
    ([4], "int8_ef"), ([4], "bf16_each"), ([4], 9), ([4, 4], "fp32", [0, 3]), ([4], "fp32", [1 << 62]), ([1 << 41], "fp32"),
    ([1 << 40, 1], "fp32"), ([5, 5], "bf16", [10, 14]),
])
def test_norm_create_refuses(args):
    refused(BAD, B.ar_norm_plan_create, *args)


def test_norm_plans():
    p = B.ar_norm_plan_create([10, 0, 500], "bf16", [3, 7, 100])  # an empty tensor may lie anywhere
    s = B.ar_norm_plan_stats(p)
    assert (s["ntensors"], s["device"], s["grad_bytes"], s["count"], s["arena_count"]) == (3, -1, 2, 510, 600)
    assert s["workspace_bytes"] > 0
    B.ar_norm_plan_destroy(p)
    p = B.ar_norm_plan_create([], "fp32")
    assert B.ar_norm_plan_stats(p)["arena_count"] == 0
    B.ar_norm_plan_destroy(p)
    with pytest.raises(ValueError, match="offsets"):
        B.ar_norm_plan_create([1, 2], "fp32", [0])
    assert not B.lib().ar_norm_plan_create(-1, None, None, 0)
    assert not B.lib().ar_norm_plan_create((1 << 20) + 1, None, None, 0)
    assert not B.lib().ar_norm_plan_create(1, None, None, 0)


@pytest.mark.parametrize("change,word", [
    (dict(g=0), "grads is NULL"), (dict(g=far(0) + 1), "grads is not aligned"), (dict(n=0), "norm is NULL"),
    (dict(n=far(1) + 2), "norm is not aligned"), (dict(t=far(2) + 2), "tensor_norms is not aligned"),
    (dict(n=far(0) + 1196), "overlap"), (dict(t=far(0) - 8), "overlap"), (dict(t=far(1) - 8), "overlap"),
    (dict(scale=-1.0), "scale"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
])
def test_norm_refuses(norm, change, word):
    a = dict(g=far(0), n=far(1), t=far(2), scale=1.0) | change
    assert word in refused(BAD, B.ar_grad_norm, norm, a["g"], a["n"], a["t"], a["scale"])


@pytest.mark.parametrize("change,word", [
    (dict(g=0), "grads is NULL"), (dict(g=far(0) + 1, o=None), "grads is not aligned"), (dict(n=0), "norm is NULL"),
    (dict(o=far(2) + 1), "grads_out is not aligned"), (dict(o=far(0) + 2), "overlap"), (dict(n=far(2)), "overlap"),
    (dict(n=far(0), o=None), "overlap"), (dict(most=0.0), "max_norm"), (dict(most=-1.0), "max_norm"),
    (dict(most=float("inf")), "max_norm"), (dict(most=1e39), "max_norm"), (dict(most=float("nan")), "max_norm"),
    (dict(most=1e-50), "max_norm"),
])
def test_clip_refuses(norm, change, word):
    a = dict(g=far(0), o=far(2), n=far(1), most=1.0) | change
    assert word in refused(BAD, B.ar_grad_clip, norm, a["g"], a["n"], a["most"], a["o"])


def test_null_plans():
    refused(BAD, B.ar_grad_norm, None, far(0), far(1))
    refused(BAD, B.ar_grad_clip, None, far(0), far(1), 1.0)
    refused(BAD, B.ar_norm_plan_prepare, None)
    refused(BAD, B.ar_rmsnorm_forward, None, far(0), far(1), ntokens=1)
    refused(BAD, B.ar_rmsnorm_backward, None, *[far(i) for i in range(6)], ntokens=1)
    refused(BAD, B.ar_rmsnorm_prepare, None)
    for fn in (B.ar_qexperts_forward, B.ar_qexperts_input_grad):
        refused(BAD, fn, None, *[far(i) for i in range(6)], ntokens=1)
    refused(BAD, B.ar_qexperts_quantize, None, far(0), far(1), far(2), dtype="bf16")
    refused(BAD, B.ar_qexperts_prepare, None)
    refused(BAD, B.ar_qexperts_launch_shape, None, "forward", 1)
    L = B.lib()
    assert L.ar_rmsnorm_forward(far(0), None, 1, None) == BAD
    assert L.ar_rmsnorm_backward(far(0), None, 1, None) == BAD
    for s in (L.ar_norm_plan_stats(None), L.ar_rmsnorm_stats(None), L.ar_qexperts_stats(None)):
        assert s.device == 0 and s.workspace_bytes == 0
    B.ar_norm_plan_destroy(None)
    B.ar_rmsnorm_destroy(None)
    B.ar_qexperts_destroy(None)


# ---------------------------------------------------------------- RMS norm

@pytest.mark.parametrize("args", [
    (0, "bf16"), (65537, "bf16"), (8, "int8_ef"), (8, "bf16", "bf16_each"), (8, "fp32", "fp32", 7),
    (8, "fp32", "fp32", "fp32", -1e-6), (8, "fp32", "fp32", "fp32", 0.0), (8, "fp32", "fp32", "fp32", float("inf")), (8, "fp32", "fp32", "fp32", float("nan")),
])
def test_rmsnorm_create_refuses(args):
    refused(BAD, B.ar_rmsnorm_create, *args)


@pytest.mark.parametrize("features", [1, 300, 4096, 65536])
def test_rmsnorm_stats(features):
    p = B.ar_rmsnorm_create(features, "bf16", "fp32", "bf16")
    s = B.ar_rmsnorm_stats(p)
    B.ar_rmsnorm_destroy(p)
    assert (s["device"], s["features"], s["elem_bytes"], s["gain_bytes"], s["grad_bytes"]) == (-1, features, 2, 4, 2)
    assert 4 * features <= s["workspace_bytes"] <= 64 << 20


FWD = dict(x=far(0), gain=far(1), residual=far(2), h=far(3), y=far(4), codes=far(5), scales=far(6), rstd=far(7), ntokens=4)


@pytest.mark.parametrize("change,word", [
    (dict(x=0), "x is NULL"), (dict(x=far(0) + 1), "x is not aligned"), (dict(gain=0), "gain is NULL"),
    (dict(gain=far(1) + 2), "gain is not aligned"), (dict(residual=far(2) + 1), "residual is not aligned"),
    (dict(h=far(3) + 1), "h is not aligned"), (dict(y=far(4) + 1), "y is not aligned"), (dict(rstd=far(7) + 2), "rstd is not aligned"),
    (dict(codes=None), "together"), (dict(scales=None), "together"), (dict(strides={"x": 299}), "x: row stride"),
    (dict(strides={"residual": 299}), "residual: row stride"), (dict(strides={"h": 299}), "h: row stride"),
    (dict(strides={"y": (1 << 22) + 1}), "y: row stride"), (dict(strides={"codes": 299}), "codes: row stride"),
    (dict(strides={"scales": 2}), "scales: row stride"), (dict(ntokens=1 << 31), "tokens"),
    (dict(h=far(0) + 600), "h and x overlap"), (dict(h=far(0), strides={"h": 304}), "h and x overlap"),
    (dict(y=far(2) + 2), "y and residual overlap"), (dict(y=far(3)), "y and h overlap"), (dict(codes=far(0)), "codes and x"),
    (dict(codes=far(4)), "codes and y"), (dict(scales=far(5) + 8), "scales and codes"), (dict(rstd=far(1)), "rstd and gain"),
    (dict(rstd=far(0)), "rstd and x"), (dict(h=far(1)), "h and gain"),
])
def test_rmsnorm_forward_refuses(rms, change, word):
    assert word in refused(BAD, B.ar_rmsnorm_forward, rms, **(FWD | change))


BWD = dict(dy=far(0), h=far(1), gain=far(2), rstd=far(3), dx=far(4), dgain=far(5), dh=far(6), ntokens=4)


@pytest.mark.parametrize("change,word", [
    (dict(dy=0), "dy is NULL"), (dict(h=0), "h is NULL"), (dict(gain=0), "gain is NULL"), (dict(rstd=0), "rstd is NULL"),
    (dict(dx=0), "dx is NULL"), (dict(dgain=0), "dgain is NULL"), (dict(dgain=far(5) + 2), "dgain is not aligned"),
    (dict(dy=far(0) + 1), "dy is not aligned"), (dict(dh=far(6) + 1), "dh is not aligned"), (dict(ntokens=1 << 31), "tokens"),
    (dict(strides={"dy": 299}), "dy: row stride"), (dict(strides={"dh": 299}), "dh: row stride"), (dict(strides={"h": 299}), "h: row stride"),
    (dict(strides={"dx": 299}), "dx: row stride"), (dict(dx=far(0) + 2), "dx and dy overlap"),
    (dict(dx=far(1), strides={"dx": 301}), "dx and h overlap"), (dict(dx=far(6) + 600), "dx and dh overlap"),
    (dict(dgain=far(4)), "dgain and dx"), (dict(dgain=far(2)), "dgain and gain"), (dict(dx=far(3)), "dx and rstd"),
    (dict(dgain=far(0)), "dgain and dy"), (dict(ntokens=0, dgain=0), "dgain is NULL"),
])
def test_rmsnorm_backward_refuses(rms, change, word):
    assert word in refused(BAD, B.ar_rmsnorm_backward, rms, **(BWD | change))


# ------------------------------------------------- 8-bit rows and products

@pytest.mark.parametrize("change,word", [
    (dict(dtype="int8_ef"), "AR_FLOAT32"), (dict(features=0), "features"), (dict(features=(1 << 22) + 1), "features"),
    (dict(ntokens=1 << 31), "tokens"), (dict(x=0), "x is NULL"), (dict(x=far(0) + 1), "x is not aligned"),
    (dict(codes=0), "codes is NULL"), (dict(scales=0), "scales is NULL"), (dict(x_stride=299), "x: row stride"),
    (dict(codes_stride=299), "codes: row stride"), (dict(scales_stride=2), "scales: row stride"),
    (dict(codes=far(0)), "overlap"), (dict(scales=far(0)), "overlap"), (dict(scales=far(1) + 1), "overlap"),
])
def test_quantize_rows_refuses(change, word):
    a = dict(x=far(0), codes=far(1), scales=far(2), dtype="bf16", features=300, ntokens=4) | change
    assert word in refused(BAD, B.ar_quantize_rows, **a)


def test_quantize_no_rows():
    B.ar_quantize_rows(0, 0, 0, dtype="fp32", features=5, ntokens=0)
    with pytest.raises(ValueError, match="address"):
        B.ar_quantize_rows(far(0), far(1), far(2))
    with pytest.raises(ValueError, match="not a device tensor"):
        B.ar_quantize_rows(torch.zeros(2, 3), far(1), far(2))


@pytest.mark.parametrize("args", [
    (0, 64, 64, "bf16"), (65537, 64, 64, "bf16"), (4, 0, 64, "bf16"), (4, 64, (1 << 22) + 1, "bf16"), (4, 64, 64, "int8_ef"),
    (2, 4, 4, "bf16", [0, 15]), (2, 4, 4, "bf16", [0, 1 << 62]),
])
def test_qexperts_create_refuses(args):
    refused(BAD, B.ar_qexperts_create, *args)


def test_qexperts_stats():
    p = B.ar_qexperts_create(3, 300, 129, "fp32", [100, 60000, 200000])
    s = B.ar_qexperts_stats(p)
    B.ar_qexperts_destroy(p)
    assert s == {"nexperts": 3, "device": -1, "in_features": 300, "out_features": 129, "elem_bytes": 4,
                 "arena_count": 200000 + 300 * 129, "scale_count": 3 * 2 * 3, "workspace_bytes": 3 * 8}
    with pytest.raises(ValueError, match="weight offsets"):
        B.ar_qexperts_create(3, 4, 4, "bf16", [0, 16])


@pytest.mark.parametrize("change,word", [
    (dict(x=0), "x is NULL"), (dict(xs=0), "x_scales is NULL"), (dict(w=0), "arena is NULL"), (dict(ws=0), "weight_scales is NULL"),
    (dict(y=0), "y is NULL"), (dict(y=far(4) + 1), "y is not aligned"), (dict(ends=0), "ends is NULL"),
    (dict(ends=far(5) + 2), "ends is not aligned"), (dict(x_stride=299), "x: row stride"), (dict(x_scales_stride=2), "x_scales: row stride"),
    (dict(y_stride=199), "y: row stride"), (dict(y=far(0) + 8), "y and x overlap"), (dict(y=far(1)), "y and x_scales overlap"),
    (dict(y=far(2) + 100), "overlap"), (dict(y=far(3)), "y and weight_scales overlap"), (dict(y=far(5)), "y and ends overlap"),
    (dict(n=1 << 31), "tokens"),
])
def test_qexperts_forward_refuses(experts, change, word):
    a = dict(x=far(0), xs=far(1), w=far(2), ws=far(3), y=far(4), ends=far(5), n=8) | change
    kw = {k: v for k, v in a.items() if k.endswith("_stride")}
    assert word in refused(BAD, B.ar_qexperts_forward, experts, a["x"], a["xs"], a["w"], a["ws"], a["y"], a["ends"],
                           ntokens=a["n"], **kw)


@pytest.mark.parametrize("change,word", [
    (dict(x=0), "dy is NULL"), (dict(y=far(4) + 1), "dx is not aligned"), (dict(dy_stride=199), "dy: row stride"),
    (dict(dy_scales_stride=1), "dy_scales: row stride"), (dict(dx_stride=299), "dx: row stride"), (dict(y=far(0)), "dx and dy overlap"),
])
def test_qexperts_input_grad_refuses(experts, change, word):
    a = dict(x=far(0), xs=far(1), w=far(2), ws=far(3), y=far(4), ends=far(5), n=8) | change
    kw = {k: v for k, v in a.items() if k.endswith("_stride")}
    assert word in refused(BAD, B.ar_qexperts_input_grad, experts, a["x"], a["xs"], a["w"], a["ws"], a["y"], a["ends"],
                           ntokens=a["n"], **kw)


@pytest.mark.parametrize("change,word", [
    (dict(w=0), "arena is NULL"), (dict(w=far(0) + 2), "not aligned"), (dict(c=0), "codes is NULL"), (dict(s=0), "scales is NULL"),
    (dict(c=far(0) + 4), "overlap"), (dict(s=far(1) + 7), "overlap"), (dict(s=far(0)), "overlap"), (dict(dtype="bf16_each"), "AR_FLOAT32"),
])
def test_qexperts_quantize_refuses(experts, change, word):
    a = dict(w=far(0), c=far(1), s=far(2), dtype="fp32") | change
    assert word in refused(BAD, B.ar_qexperts_quantize, experts, a["w"], a["c"], a["s"], dtype=a["dtype"])


def test_qexperts_launch_shape(experts):
    assert B.ar_qexperts_launch_shape(experts, "forward", 0) == {"tile_rows": 0, "tile_cols": 0}
    for product in ("forward", "input_grad"):
        for n in (1, 100, 5000):
            s = B.ar_qexperts_launch_shape(experts, product, n)
            assert s["tile_rows"] > 0 and s["tile_cols"] > 0
    refused(BAD, B.ar_qexperts_launch_shape, experts, "weight_grad", 5)
    refused(BAD, B.ar_qexperts_launch_shape, experts, "forward", 1 << 31)


def test_binding_checks_tensors(rms, experts, norm):
    x = torch.zeros(4, 300, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not a device tensor"):
        B.ar_rmsnorm_forward(rms, x, far(1), y=far(2))
    with pytest.raises(ValueError, match="ntokens"):
        B.ar_rmsnorm_forward(rms, far(0), far(1), y=far(2))
    with pytest.raises(ValueError, match="own stride"):
        B.ar_rmsnorm_forward(rms, x, far(1), y=far(2), strides={"x": 300})
    with pytest.raises(ValueError, match="not a device tensor"):
        B.ar_qexperts_forward(experts, torch.zeros(4, 300, dtype=torch.uint8), *[far(i) for i in range(5)])
    with pytest.raises(ValueError, match="address"):
        B.ar_qexperts_quantize(experts, far(0), far(1), far(2))
    with pytest.raises(ValueError, match="not a device tensor"):
        B.ar_grad_norm(norm, torch.zeros(600, dtype=torch.bfloat16), far(1))


def test_binding_refuses_unknown_strides(rms):
    with pytest.raises(ValueError, match="strides of"):
        B.ar_rmsnorm_forward(rms, far(0), far(1), y=far(2), ntokens=4, strides={"code": 300})
    with pytest.raises(ValueError, match="strides of"):
        B.ar_rmsnorm_backward(rms, far(0), far(1), far(2), far(3), far(4), far(5), ntokens=4, strides={"y": 300})


def test_structs_are_as_the_header_has_them(tmp_path):
    """Sizes of the structs that cross the ABI, from a C compiler."""
    import os
    import subprocess

    src = tmp_path / "s.c"
    names = ("ar_norm_stats_t", "ar_rmsnorm_stats_t", "ar_rmsnorm_forward_t", "ar_rmsnorm_backward_t", "ar_qexperts_stats_t")
    src.write_text('#include "ar.h"\n#include <stdio.h>\nint main(void){' +
                   "".join(f'printf("%zu\\n", sizeof({n}));' for n in names) + "return 0;}\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    sizes = [int(v) for v in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()]
    assert sizes == [ctypes.sizeof(getattr(B, n)) for n in names]
    for packed, fields in ((B._FORWARD, B.ar_rmsnorm_forward_t), (B._BACKWARD, B.ar_rmsnorm_backward_t)):
        values = list(range(1, len(fields._fields_) + 1))
        assert packed.size == ctypes.sizeof(fields)
        made = fields.from_buffer_copy(packed.pack(*values))
        assert [getattr(made, k) for k, _ in fields._fields_] == values


def test_rmsnorm_forward_needs_no_workspace(rms):
    """No rows: done, without a device to prepare the plan on."""
    B.ar_rmsnorm_forward(rms, far(0), far(1), y=far(2), ntokens=0)
    assert B.ar_rmsnorm_stats(rms)["device"] == -1


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("counts", [[1 << 40], [1 << 37, 1 << 38, 5], [(1 << 20) - 1] * (1 << 20)], ids=["one", "three", "many"])
def test_norm_plans_fit_a_launch(counts, dtype):
    """Every plan within the documented limits has its chunks, a wave each and 8 to a workgroup of 512 threads, in one
    launch (less than 2^31 threads).  A chunk takes 16 bytes of the workspace, and 8 of sums, its workgroup 8 more, a
    tensor 4."""
    p = B.ar_norm_plan_create(counts, dtype)
    n = B.ar_norm_plan_stats(p)["workspace_bytes"] - 4 * (len(counts) + 1)
    B.ar_norm_plan_destroy(p)
    assert n / 25 < (1 << 31) // 64


def test_norm_create_refuses_before_it_builds():
    """Overlapping tensors are refused without the memory that their chunks would take."""
    import subprocess
    import sys

    code = """
import resource
from gradient_all_reduce_ar_amd import _binding as B
B.lib()
pages = int(open("/proc/self/statm").read().split()[0])
resource.setrlimit(resource.RLIMIT_AS, (pages * resource.getpagesize() + (64 << 20),) * 2)
try:
    B.ar_norm_plan_create([1 << 39, 1 << 39], "fp32", [0, 5])
except B.ArError as e:
    print(e)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100)
    assert "tensors overlap" in r.stdout, r.stdout + r.stderr
