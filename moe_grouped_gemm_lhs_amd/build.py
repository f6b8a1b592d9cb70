"""Build libdg.so in-tree for gfx950 with hipcc, and the Python module _marshal beside it.

Run ``python -m moe_grouped_gemm_lhs_amd.build`` (or call ``build()``).  Every HIP
translation unit is compiled with packed fp32 VALU ops disabled; hipcc's host pass
warns that it does not know that feature, which is harmless."""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libdg.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["dg_kernels.hip", "dg_quant.hip", "dg_noalloc.hip", "dg_route.hip", "dg_lora.hip",
           "dg_host.cpp", "dg_ops_host.cpp"]
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA results straight into VGPRs, where the promotion FMAs read them
    "-mllvm", "-amdgpu-mfma-vgpr-form=1",
    "-I", INCLUDE, "-I", CSRC,
]


def build(verbose: bool = False) -> str:
    """Compile every source and link libdg.so, then _marshal.so (always rebuilds)."""
    objs = []
    for src in SOURCES:
        obj = os.path.join(CSRC, f"{src}.{os.getpid()}.o")
        cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        objs.append(obj)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    for o in objs:
        os.remove(o)
    build_marshal(verbose)
    return LIB


def build_marshal(verbose: bool = False) -> str:
    """Host code only, by the one compiler, against libdg.so and the headers of torch and Python."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths

    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [HIPCC, "-no-hip-rt", "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-isystem", sysconfig.get_paths()["include"]]
    for path in include_paths():
        cmd += ["-isystem", path]
    cmd += [os.path.join(CSRC, "dg_marshal.cpp"), "-o", tmp, "-L", PKG, "-l:libdg.so",
            "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu",
            "-lc10", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, MARSHAL)
    return MARSHAL


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
