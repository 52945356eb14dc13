"""Build libmxmoe.so (HIP kernels + C ABI) for gfx950 with hipcc, and _nodes.so
(autograd nodes over it, C++ against the installed torch), in-tree.

Usage: python -m mxfp8_block_scaled_06_amd.build
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libmxmoe.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
NODES_NAME = "_nodes.so"

SOURCES = ["mx_quant.hip", "mx_gemm.hip", "mx_route.hip", "mx_noalloc.hip", "mx_fp4.hip", "mx_fp4_gemm.hip", "mx_moe.hip",
           "mx_router.hip", "mx_swiglu.hip", "mx_combine.hip", "mx_api.cpp"]

# -packed-fp32-ops: never emit packed fp32 VALU instructions.
HIP_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: install ROCm or put hipcc on PATH")


def _nodes_commands(obj, out):
    """Compile and link _nodes.so: host C++ only; libmxmoe.so is found beside it."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("g++ not found: the autograd nodes need a C++ compiler")
    include = [*include_paths(), sysconfig.get_paths()["include"], "/opt/rocm/include", INCLUDE]
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-w", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in include),
                "-c", os.path.join(CSRC, "mx_nodes.cpp"), "-o", obj]
    link = [cxx, "-shared", obj, "-o", out, f"-L{lib}", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip", "-ltorch_python",
            f"-L{PKG}", f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def _run(cmd):
    proc = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in proc.stdout.splitlines() if "packed-fp32-ops" not in l)
    if proc.returncode != 0:
        raise RuntimeError(f"command failed ({proc.returncode}): {' '.join(cmd)}\n{out}")
    return out


def build(verbose: bool = False) -> str:
    cc = hipcc()
    with tempfile.TemporaryDirectory(prefix="mxmoe_build_") as tmp:
        objs = []
        cmds = []
        for src in SOURCES:
            obj = os.path.join(tmp, src + ".o")
            lang = ["-x", "hip"] if src.endswith(".hip") else []
            cmds.append([cc, *HIP_FLAGS, "-I", INCLUDE, "-I", CSRC, *lang, "-c", os.path.join(CSRC, src), "-o", obj])
            objs.append(obj)
        nodes = os.path.join(tmp, NODES_NAME)
        compile_nodes, link_nodes = _nodes_commands(os.path.join(tmp, "mx_nodes.o"), nodes)
        cmds.append(compile_nodes)
        with ThreadPoolExecutor(max_workers=len(cmds)) as ex:
            for out in ex.map(_run, cmds):
                if verbose and out.strip():
                    print(out)
        tmp_lib = os.path.join(tmp, LIB_NAME)
        _run([cc, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp_lib])
        shutil.move(tmp_lib, LIB_PATH)
        _run(link_nodes)
        shutil.move(nodes, os.path.join(PKG, NODES_NAME))
    if verbose:
        print(f"built {LIB_PATH} and {NODES_NAME}")
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
