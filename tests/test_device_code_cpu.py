"""The device code that the compiler makes of the kernels' building blocks
(compiled for gfx950, not run)."""
import os
import re
import subprocess

import pytest

from gradient_all_reduce_ar_amd import build as libbuild

HIPCC = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")

BETWEEN = """
#include "tiles.hpp"
using Lds = __attribute__((address_space(3))) float;
using Global = const __attribute__((address_space(1))) float;
extern "C" __global__ void between(const float *g, ar_dev::ux4 r, unsigned off, float *out) {
  __shared__ float a[128], b[256];
  const uint32_t to = __builtin_amdgcn_readfirstlane(ar_dev::lds_offset(b));
  __builtin_amdgcn_global_load_lds((Global *)(g + threadIdx.x), (Lds *)a, 4, 0, 0);
  ar_dev::load_to_lds(r, off, to);
  __builtin_amdgcn_global_load_lds((Global *)(g + 64 + threadIdx.x), (Lds *)a, 4, 256, 0);
  __syncthreads();
  out[threadIdx.x] = a[threadIdx.x] + b[threadIdx.x];
}
"""


def assembly(source, tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not installed")
    src, out = tmp_path / "k.hip", tmp_path / "k.s"
    src.write_text(source)
    flags = [f for f in libbuild.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    r = subprocess.run([HIPCC, *flags, "--cuda-device-only", "-S", "-I", libbuild.CSRC, str(src), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out.read_text()


def test_the_compiler_knows_that_a_load_to_the_lds_changes_m0(tmp_path):
    """m0 says where such a load goes in the LDS.  One of the compiler's own behind load_to_lds sets it again,
    though it had the same value before."""
    text = assembly(BETWEEN, tmp_path)
    behind = text[text.index("buffer_load_dwordx4"):]
    before_next = behind[:behind.index("global_load_lds")]
    assert re.search(r"s_mov\w* m0,", before_next), before_next
