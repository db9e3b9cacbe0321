"""Builds libar.so (the HIP kernels, planner and C ABI) for gfx950, in-tree."""
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libar.so")
# Host code instrumented with AddressSanitizer and UndefinedBehaviorSanitizer
# (device code unchanged), for the CPU tests of the planner and the C ABI.
# Load it with AR_LIB=<path> and the clang ASan runtime preloaded.
LIB_SANITIZED = os.path.join(HERE, "libar_sanitized.so")
SANITIZE_FLAGS = "-Xarch_host -fsanitize=address -Xarch_host -fsanitize=undefined " \
                 "-Xarch_host -fno-sanitize-recover=undefined -Xarch_host -fno-omit-frame-pointer".split()
SOURCES = ["plan.cpp", "kernels.hip", "qkernels.hip", "capi.hip", "experts.hip", "muon.hip", "qexperts.hip",
           "rmsnorm.hip", "clip.hip", "oapi.hip", "tapi.hip"]

# -ffp-contract=off and no fast-math: every add is one IEEE binary32 add.
# -fno-gpu-flush-denormals-to-zero: fp32 denormals are kept on the device.
# packed-fp32 ops are disabled: the kernels are built from scalar adds.
# fp32 division on the device is correctly rounded (the INT8 quantizer).
HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-ffp-contract=off", "-fno-fast-math", "-fno-gpu-flush-denormals-to-zero",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd))
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("hipcc failed")
    # the host pass does not know the packed-fp32 feature and says so; drop that noise
    noise = "'-packed-fp32-ops' is not a recognized feature"
    for line in (r.stdout + r.stderr).splitlines():
        if noise not in line and line.strip() and verbose:
            print(line)


def build(out=LIB, defines=(), verbose=False, sanitize=False):
    """Compiles every source, several at a time, and links them."""
    hipcc = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")
    os.makedirs(os.path.join(HERE, "_build"), exist_ok=True)
    flags = [*HIPCC_FLAGS, *(SANITIZE_FLAGS if sanitize else []), *[f"-D{d}" for d in defines]]
    with tempfile.TemporaryDirectory(dir=os.path.join(HERE, "_build")) as tmp:
        def compiled(source):
            obj = os.path.join(tmp, source + ".o")
            _run([hipcc, *[f for f in flags if f != "-shared"], "-c", "-o", obj, os.path.join(CSRC, source)], verbose)
            return obj

        with ThreadPoolExecutor(max(1, min(8, int(os.environ.get("MAX_JOBS") or 8)))) as pool:
            objs = list(pool.map(compiled, SOURCES))
        _run([hipcc, *flags, "-o", out, *objs], verbose)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
