"""Build libmoe.so (HIP, gfx950) in-tree with hipcc, and the small Python
module _bind in front of its linear operators.

Usage: python -m moe_expert_layer_sigmoid_amd.build  (or build() from Python).
Every HIP source is compiled with packed-fp32 instruction selection turned
off (-Xclang -target-feature -Xclang -packed-fp32-ops).
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmoe.so")
BIND = os.path.join(PKG, "_bind.so")
SOURCES = ["moe_api.hip", "kernels_front.hip", "kernels_gemm.hip", "kernels_tiled.hip", "eplb.hip",
           "kernels_router.hip", "kernels_a16.hip", "linear_api.hip", "kernels_linear.hip",
           "kernels_fp8_quant.hip", "kernels_linear_act.hip", "kernels_linear_act_f16.hip",
           "kernels_act_backward.hip", "kernels_grad.hip", "kernels_a16w16.hip"]
ARCH = os.environ.get("MOE_OFFLOAD_ARCH", "gfx950")


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def flags():
    return [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _run(cmd, verbose: bool, what: str) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")


def _build_bind(verbose: bool) -> None:
    """_bind.so: CPython module in front of libmoe, against torch's headers."""
    import torch
    from torch.utils.cpp_extension import include_paths

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    inc = [*include_paths(), sysconfig.get_paths()["include"], os.path.join(rocm, "include"), os.path.join(ROOT, "include")]
    tmp = BIND + ".tmp"
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          f'-DMOE_TORCH_VERSION="{torch.__version__}"', *(a for p in inc for a in ("-isystem", p)),
          os.path.join(CSRC, "bind.cpp"), "-o", tmp, LIB, f"-L{lib}", "-lc10", "-lc10_hip", "-ltorch_cpu",
          "-ltorch_python", "-Wl,-rpath,$ORIGIN"], verbose,
         "bind.cpp (libmoe.so is built and complete: without _bind the linear calls are checked in Python)")
    os.replace(tmp, BIND)


def build(verbose: bool = False) -> str:
    objs = [os.path.join(CSRC, src.replace(".hip", ".o")) for src in SOURCES]
    jobs = sorted(zip(SOURCES, objs), key=lambda so: "linear" not in so[0])   # the longest first
    with ThreadPoolExecutor(4) as ex:
        list(ex.map(lambda so: _run([hipcc(), *flags(), "-c", os.path.join(CSRC, so[0]), "-o", so[1]], verbose, so[0]), jobs))
    tmp = LIB + ".tmp"
    _run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,-soname,libmoe.so", "-o", tmp, *objs], verbose, "link")
    os.replace(tmp, LIB)
    for o in objs:
        os.remove(o)
    _build_bind(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
