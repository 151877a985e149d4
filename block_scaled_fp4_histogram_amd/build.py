"""Builds the gfx950 library block_scaled_fp4_histogram_amd/libmoe_gfx950.so with hipcc, and the torch
binding of its products (_products.so) with the host compiler."""
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmoe_gfx950.so")
SOURCES = [os.path.join(CSRC, "moe_kernels.hip"), os.path.join(CSRC, "moe_decode.hip"),
           os.path.join(CSRC, "moe_prefill.hip"), os.path.join(CSRC, "moe_static.hip"),
           os.path.join(CSRC, "moe_mm.hip"), os.path.join(CSRC, "moe_rows.hip"),
           os.path.join(CSRC, "moe_api.cpp"), os.path.join(CSRC, "moe_mm_api.cpp")]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # an entry point that references a missing definition fails here, not at load time
    "-Wl,--no-undefined",
    "-munsafe-fp-atomics",
    # MFMA accumulators in VGPRs: in-place accumulation, no AGPR copies in pipelined loops
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    # packed fp32 VALU forms are kept out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


BINDING = os.path.join(PKG, "_products.so")


def build_binding(verbose: bool = False) -> str:
    """The torch binding of the products: host code only. The library, and the layer through it, do without."""
    import sysconfig
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", os.path.join(ROOT, "include")]
    for d in include_paths() + [sysconfig.get_paths()["include"]]:
        cmd += ["-isystem", d]
    cmd += [os.path.join(CSRC, "moe_torch.cpp"), "-o", BINDING + ".tmp"]
    for d in library_paths():
        cmd += ["-L", d]
    cmd += ["-lc10", "-ltorch", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"building the binding failed: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"building the binding failed ({r.returncode}):\n{r.stderr}")
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build(verbose: bool = False) -> str:
    """The library."""
    cmd = [HIPCC] + FLAGS + SOURCES + ["-o", LIB + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "packed-fp32-ops"
    err = "\n".join(l for l in (r.stderr or "").splitlines() if noise not in l and l.strip())
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed ({r.returncode}):\n{err}")
    if verbose and err:
        print(err, file=sys.stderr)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    build_binding(verbose=True)
