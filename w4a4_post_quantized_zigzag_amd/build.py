"""Build libw4a4.so in-tree with hipcc for gfx950, and the torch-facing marshalling of the single-token
calls beside it where torch and a C++ compiler are there (python -m w4a4_post_quantized_zigzag_amd.build)."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libw4a4.so")
SOURCES = ["abi.hip", "k_pack.hip", "k_act.hip", "k_gemm.hip", "k_calib.hip", "k_gptq.hip",
           "k_w4g.hip", "k_decode.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# Device code is built without packed-fp32 instructions (v_pk_*_f32); every unit is gfx950-only.
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]
# Per-unit extras: the activation kernels keep MFMA accumulators in ordinary VGPRs (their results
# feed VALU work right away, so the accumulation-register form would only add copies).
EXTRA_FLAGS = {"k_act.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
               "k_decode.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, *EXTRA_FLAGS.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _lacks_for_marshalling() -> str | None:
    """What this machine lacks for _decode.so (the library itself needs hipcc alone), or None."""
    try:
        from torch.utils.cpp_extension import include_paths
    except ImportError as e:
        return f"torch ({e})"
    cxx = os.environ.get("CXX", "g++")
    if shutil.which(cxx) is None:
        return f"the C++ compiler {cxx}"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    if not any(os.path.exists(os.path.join(p, "c10", "hip", "HIPStream.h")) for p in include_paths()):
        return "torch's HIP headers"
    return None


def _build_marshalling(out: str) -> None:
    """_decode.so: host code against torch's headers and the library just linked beside it."""
    import torch
    from torch.utils.cpp_extension import ROCM_HOME, include_paths
    rocm = ROCM_HOME or os.path.dirname(os.path.dirname(shutil.which(HIPCC) or HIPCC))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-D__HIP_PLATFORM_AMD__=1",
           "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(rocm, "include"),
           "-isystem", sysconfig.get_paths()["include"]]
    for p in include_paths():
        cmd += ["-isystem", p]
    cmd += [os.path.join(CSRC, "py_decode.cpp"), "-o", out + ".tmp", LIB,
            "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu",
            "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{LIB} is complete, but the marshalling build failed:\n{r.stdout}\n{r.stderr}")
    os.replace(out + ".tmp", out)


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-Wl,-soname,libw4a4.so", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    mod = os.path.join(PKG, "_decode.so")
    if os.path.exists(mod):  # it belongs to the library that was just replaced
        os.remove(mod)
    lacks = _lacks_for_marshalling()
    if lacks is None:
        _build_marshalling(mod)
    if verbose:
        print(f"built {LIB} and {mod}" if lacks is None else
              f"built {LIB}; without {lacks} the single-token calls have no Python side ({mod})")
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
