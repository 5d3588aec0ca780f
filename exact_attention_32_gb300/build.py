"""Build libfa.so (the CUDA library behind include/fa.h) in-tree for sm_103a.

Each .cu under csrc/ is compiled by nvcc in parallel, then linked into
``exact_attention_32_gb300/libfa.so`` (static CUDA runtime); the binding's
extension ``_marshal.so`` by g++ against the installed torch.  ptxas resource
reports (registers, spills, shared memory) are kept next to the objects in
``_build/<name>.ptxas.txt``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfa.so")
MARSHAL_SRC = os.path.join(PKG, "_marshal.cpp")
MARSHAL = os.path.join(PKG, "_marshal.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def _compile(src: str) -> str:
    name = os.path.splitext(os.path.basename(src))[0]
    obj = os.path.join(BUILD, name + ".o")
    r = subprocess.run([nvcc()] + NVCC_FLAGS + ["-c", src, "-o", obj],
                       capture_output=True, text=True)
    with open(os.path.join(BUILD, name + ".ptxas.txt"), "w") as f:
        f.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build_marshal(force: bool = False) -> str:
    """Compile the binding's extension unless it is newer than its sources and was built with this torch."""
    import torch

    deps = [MARSHAL_SRC, os.path.join(INCLUDE, "fa.h"), __file__]
    stamp, made_with = os.path.join(BUILD, "_marshal.torch.txt"), None
    if os.path.exists(stamp):
        with open(stamp) as f:
            made_with = f.read()
    if (not force and made_with == torch.__version__ and os.path.exists(MARSHAL)
            and os.path.getmtime(MARSHAL) >= max(os.path.getmtime(p) for p in deps)):
        return MARSHAL
    os.makedirs(BUILD, exist_ok=True)
    tmp, at = MARSHAL + ".tmp", os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(at, "include"),
           os.path.join(at, "include", "torch", "csrc", "api", "include"), cuda]
    r = subprocess.run([shutil.which("g++") or "c++", "-O2", "-std=c++17", "-shared", "-fPIC"] +
                       [x for i in inc for x in ("-isystem" if i != INCLUDE else "-I", i)] +
                       [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", MARSHAL_SRC, "-o", tmp,
                        "-L", os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {MARSHAL_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return MARSHAL


def _extension(force: bool) -> None:
    try:
        import torch  # noqa: F401
    except ImportError:
        print("torch is not there: the Python calls of the 4-bit cache (_marshal.so) are not built", file=sys.stderr)
    else:
        build_marshal(force)


def _library(force: bool) -> None:
    if (not force and os.path.exists(LIB)
            and os.path.getmtime(LIB) >= max(os.path.getmtime(p) for p in _deps())):
        return
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    r = subprocess.run([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs,
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False) -> str:
    """Compile and link libfa.so, and compile the extension beside it, unless newer than every source.

    The library needs nvcc alone: it is there whatever becomes of the
    extension, which is left out, with a note, where torch cannot be imported
    (C callers); what else goes wrong with it raises once the library is linked."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        extension = ex.submit(_extension, force)
        _library(force)
        extension.result()
    return LIB


if __name__ == "__main__":
    print(build(force=True))
