"""Build the HIP library libfp8mi.so in-tree for gfx950 with hipcc, and the
extension module _fp8mi_torch.so that calls it with torch tensors.

Usage: python -m fp8_scaled_matmul_amd.build   (or call build()).  The library
needs hipcc alone; the extension module torch and g++, too.  Where those are
not there, the library is built all the same and the error says so.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfp8mi.so")
BINDING = os.path.join(PKG, "_fp8mi_torch.so")

SOURCES = ["quantize.hip", "gemm.hip", "gemm_persistent.hip", "gemm_astat.hip", "mx4_quantize.hip", "mx4_gemm.hip",
           "mx4_moe.hip", "cross_entropy.hip", "moe_route.hip", "dropout.hip", "api.cpp"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # bit-exact quantization: no FMA contraction behind the source's back
    "-ffp-contract=off",
    # packed fp32 VALU ops stay off (v_pk_{add,mul,fma}_f32 are never emitted)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


# Per-file extras.  The block-scaled GEMM promotes each MFMA result on the
# VALU: MFMA results written straight to VGPRs save a copy out of AGPRs.
EXTRA = {"gemm.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
         # the A-stationary kernel's unit loop must unroll fully (its register
         # rings are indexed by the step)
         "gemm_astat.hip": ["-mllvm", "-pragma-unroll-threshold=1000000"]}


def _compile(src: str) -> str:
    os.makedirs(BUILD, exist_ok=True)
    obj = os.path.join(BUILD, src + ".o")
    path = os.path.join(CSRC, src)
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    cmd = [HIPCC, *FLAGS, *EXTRA.get(src, []), *lang, "-c", path, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _hip_include() -> str:
    """HIP's headers, from the compiler's place; HIPCC may be a name on PATH."""
    hipcc = os.path.realpath(shutil.which(HIPCC) or HIPCC)
    return os.path.join(os.path.dirname(os.path.dirname(hipcc)), "include")


def _compile_binding() -> str:
    import torch
    os.makedirs(BUILD, exist_ok=True)
    obj = os.path.join(BUILD, "binding.cpp.o")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-Wall", "-DUSE_ROCM", "-D__HIP_PLATFORM_AMD__",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", os.path.join(ROOT, "include"),
           "-isystem", inc, "-isystem", _hip_include(),
           "-isystem", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link(cmd: list, out: str) -> None:
    tmp = out + ".tmp"
    r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    _link(["g++", "-shared", "-fPIC", obj, "-L", PKG, "-l:libfp8mi.so", "-Wl,-rpath,$ORIGIN", "-L", libs,
           "-ltorch_python", "-ltorch_cpu", "-lc10_hip", "-lc10"], BINDING)


def build(verbose: bool = False) -> str:
    """Compile every HIP/C++ source and link libfp8mi.so, then the extension
    module (always rebuilds)."""
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, SOURCES))
        _link([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs], LIB)
        try:
            _link_binding(binding.result())
        except Exception as e:
            raise RuntimeError(f"{LIB} is built, but not its extension module: {e}") from e
    if verbose:
        print("built", LIB, BINDING)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
