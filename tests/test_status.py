"""How the kernels' status words make the one that fa_get_device_status returns (csrc/fa_status.h, host code)."""
import ctypes
import itertools
import shutil
import subprocess

import pytest

from exact_attention_32_gb300 import build as fa_build

LAUNCH, TIMEOUT, BAD_PAGE, BAD_SEQUENCE = 5, 6, 8, 9


@pytest.fixture(scope="module")
def joined(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    at = tmp_path_factory.mktemp("status")
    (at / "t.cpp").write_text('#include "fa_status.h"\n'
                              'extern "C" int joined(const int *w, int n) { return fa_joined_status(w, n); }\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", fa_build.CSRC, "-I", fa_build.INCLUDE, str(at / "t.cpp"), "-o",
                    str(at / "t.so")], check=True)
    lib = ctypes.CDLL(str(at / "t.so"))
    return lambda *w: lib.joined((ctypes.c_int * len(w))(*w), len(w))


def test_a_wait_that_gave_up_is_not_lost_behind_a_bad_page(joined):
    # reading clears every word, so the one that says that outputs are incomplete has to be the one that is returned
    for words in itertools.permutations((0, BAD_PAGE, TIMEOUT, BAD_SEQUENCE)):
        assert joined(*words) == TIMEOUT
    for words in itertools.permutations((TIMEOUT, BAD_PAGE, LAUNCH, 0)):
        assert joined(*words) == LAUNCH


def test_otherwise_the_first_one_that_says_something(joined):
    assert joined(0, 0, 0) == 0
    assert joined(0, BAD_PAGE, 0, BAD_SEQUENCE) == BAD_PAGE and joined(BAD_SEQUENCE, 0, BAD_PAGE) == BAD_SEQUENCE
