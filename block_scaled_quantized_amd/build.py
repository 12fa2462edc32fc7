"""Build libmxgemm.so (HIP for gfx950) in-tree with hipcc.

Every source is compiled for gfx950 only, with packed-fp32 instructions disabled
(``-Xclang -target-feature -Xclang -packed-fp32-ops``). Objects go to ``_build/``; the shared
library lands next to this file, and beside it the Python binding's marshalling module (host code, against
torch's headers; left out where torch is not installed). ``python -m block_scaled_quantized_amd.build`` runs it.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import ctypes
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libmxgemm.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["api.cpp", "host_codec.cpp", "codec.hip", "mxgemm.hip", "mxgemm_ring.hip", "matvec.hip",
           "rotary.hip", "attention.hip", "pages.hip", "page_pool.cpp"]
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-x", "hip",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wno-unused-command-line-argument", f"-I{INCLUDE}", f"-I{CSRC}"]


# Per-source additions. matvec.hip: MFMA results go to ordinary VGPRs; its kernels scale every
# MFMA product on the vector ALU, and results left in accumulation registers would each need a
# v_accvgpr_read first (the GEMM kernels keep their accumulators in those registers and must not
# get this option).
EXTRA = {"matvec.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _marshal() -> str | None:
    """Compile csrc/marshal.cpp (torch's Tensor accessors, no GPU code). None, and a message, where torch, its headers,
    Python's or a host compiler are missing: the library itself needs none of them."""
    import shutil
    import sysconfig
    try:
        import torch
        home = os.path.dirname(torch.__file__)
        need = [os.path.join(home, "include", "ATen", "core", "Tensor.h"), os.path.join(sysconfig.get_paths()["include"], "Python.h")]
        missing = [p for p in need if not os.path.exists(p)] + ([] if shutil.which("g++") else ["g++"])
    except ImportError:
        missing = ["torch"]
    if missing:
        print(f"_marshal.so is not built: no {', '.join(missing)} here (the Python binding's cache calls need it; the library does not)")
        return None
    obj = os.path.join(BUILD, "marshal.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-I{INCLUDE}", f"-isystem{home}/include", f"-isystem{home}/include/torch/csrc/api/include",
           f"-isystem{sysconfig.get_paths()['include']}", "-c", os.path.join(CSRC, "marshal.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for marshal.cpp:\n{r.stderr}")
    return obj


def _link_marshal(obj: str | None) -> None:
    """The module finds libmxgemm.so beside itself; torch's libraries are those the process has loaded. One of an earlier
    build goes where there is no new one."""
    if obj is None:
        if os.path.exists(MARSHAL):
            os.remove(MARSHAL)
        return
    import torch
    tmp = MARSHAL + ".tmp"
    cmd = ["g++", "-shared", "-fPIC", obj, "-o", tmp, f"-L{HERE}", "-lmxgemm", "-Wl,-rpath,$ORIGIN",
           f"-L{os.path.dirname(torch.__file__)}/lib", "-lc10", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the marshalling module failed:\n{r.stderr}")
    os.replace(tmp, MARSHAL)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 1)) as ex:
        marshal = ex.submit(_marshal)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    # A kernel template that the host pass of hipcc fails to instantiate leaves an undefined device
    # stub behind without any diagnostic; linking a shared library lets that through, so resolve
    # every symbol now (no GPU is needed to load the library).
    try:
        ctypes.CDLL(tmp, mode=os.RTLD_NOW | os.RTLD_LOCAL)
    except OSError as e:
        raise RuntimeError(f"built library does not load: {e}") from e
    os.replace(tmp, LIB)
    _link_marshal(marshal.result())
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
