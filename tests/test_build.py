"""Sources that only the GPU tests build still compile here (nvcc cross-compiles
for sm_103a without a device), so a change to the shared headers that breaks
them fails the CPU suite rather than the GPU one."""
import ctypes
import os
import shutil
import subprocess
import sys
import tempfile

import pytest

from exact_attention_32_gb300 import build as fa_build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_tcgen05_selftest_source_compiles():
    try:
        nvcc = fa_build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    out = tempfile.mkdtemp()
    try:
        r = subprocess.run([nvcc] + fa_build.ARCH +
                           ["-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-c", "-I", fa_build.CSRC,
                            os.path.join(HERE, "cuda", "tc_selftest.cu"), "-o", os.path.join(out, "t.o")],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
    finally:
        shutil.rmtree(out, ignore_errors=True)


@pytest.mark.parametrize("missing", ["torch", "compiler"])
def test_library_is_built_without_torch_or_a_host_compiler_for_the_extension(missing, tmp_path):
    # C callers need nvcc only.  build.py as a script would run it, on one small source, with its outputs elsewhere
    try:
        fa_build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    (tmp_path / "one.cu").write_text("extern \"C\" int fa_one() { return 1; }\n")
    code = f"""
import importlib.util, os, subprocess, sys
spec = importlib.util.spec_from_file_location("b", {fa_build.__file__!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
at = {str(tmp_path)!r}
b.CSRC, b.BUILD, b.LIB = at, os.path.join(at, "_build"), os.path.join(at, "libfa.so")
b.MARSHAL = os.path.join(at, "_marshal.so")
if {missing!r} == "torch":
    sys.modules["torch"] = None  # an import of it raises ImportError
else:
    run, b.subprocess = subprocess.run, type(sys)("s")
    b.subprocess.run = lambda cmd, **kw: run(["false"] if "-ltorch_python" in cmd else cmd, **kw)
try:
    print("built", b.build())
except RuntimeError as e:
    print("raised", str(e)[:20])
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split()[0] == ("built" if missing == "torch" else "raised")
    assert ctypes.CDLL(str(tmp_path / "libfa.so")).fa_one() == 1
    assert not (tmp_path / "_marshal.so").exists()
    assert ("_marshal.so" in r.stderr) == (missing == "torch")
