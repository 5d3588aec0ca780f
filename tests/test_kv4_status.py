"""Attention over the 4-bit cache while its status word says that a wait gave up.

No wait gives up here: a copy of the kernels' source with a call that sets the
word from the host (tests/cuda/kv4_status.cu) stands in for the library.  While
the word is set the attention kernel does no work, so nothing of the call may
reach the weights, which cannot be computed again as O can.
"""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import exact_attention_32_gb300 as fa
from exact_attention_32_gb300 import build as fa_build

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "cuda", "kv4_status.cu")
FLAGS = fa_build.ARCH + ["-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-I", fa_build.CSRC, "-I", fa_build.INCLUDE]
TIMEOUT = 6


def test_source_compiles(tmp_path):
    try:
        nvcc = fa_build.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    r = subprocess.run([nvcc] + FLAGS + ["-Xptxas", "-O0", "-c", SRC, "-o", str(tmp_path / "t.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.fixture(scope="module")
def status_lib():
    out = os.path.join(HERE, "_build")
    os.makedirs(out, exist_ok=True)
    so = os.path.join(out, "libkv4status.so")
    subprocess.run([fa_build.nvcc()] + FLAGS + ["-shared", SRC, "-o", so], check=True)
    lib, p, i, i64 = ctypes.CDLL(so), ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    lib.kv4_status_decode.argtypes = [p] * 5 + [i] * 4 + [p] * 5 + [i64] * 4 + [ctypes.c_float, i, p]
    return lib


@pytest.mark.gpu
@pytest.mark.parametrize("d,G,n,n_q", [(64, 2, 100, 1), (128, 4, 100, 2), (128, 1, 4000, 1), (64, 12, 4000, 1), (128, 8, 4000, 4)])
def test_no_weight_changes_while_a_wait_is_reported(status_lib, d, G, n, n_q):
    # tables of a few tiles (whole items) and longer ones (split and merged); the workspace as an earlier call may have left it
    B, Hkv, P = 2, 2, 64
    pages = -(-n // P)
    cache = fa.kv4_cache(B * pages, Hkv, P, d)
    g = torch.Generator().manual_seed(n + d)
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(B, Hkv, n, d, generator=g).bfloat16().cuda() for _ in range(2))
    fa.kv4_append(cache, k, v, lens, table, weights=torch.rand(B, Hkv, n, generator=g).cuda())
    q = torch.randn(B, Hkv * G, n_q, d, generator=g).bfloat16().cuda()
    need = fa.fa_fwd_kv4_workspace_bytes(B, Hkv * G, Hkv, n_q, d, pages * P, True)
    scale = fa.default_scale(d)

    def call(c, ws, o, lse):
        assert status_lib.kv4_status_decode(*(t.data_ptr() for t in c), B * pages, Hkv, 6, d, q.data_ptr(), lens.data_ptr(),
                                            table.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hkv * G, n_q, pages, scale, 1,
                                            ws.data_ptr()) == 0
        torch.cuda.synchronize()

    before = [t.clone() for t in cache]
    for fill in (0, 0x3F, 0xFF):  # zeros, numbers near 0.75, NaN
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:-1], 7.0, device="cuda")
        assert status_lib.kv4_status_set(TIMEOUT) == 0
        call(cache, ws, o, lse)
        assert all(torch.equal(a, b) for a, b in zip(cache, before))
        assert (o == 7).all() and (lse == 7).all()
        assert status_lib.kv4_status_take() == TIMEOUT
    # once the word has been read the same call counts
    call(cache, ws, o, lse)
    assert status_lib.kv4_status_take() == 0
    other = fa.KV4Cache(*(t.clone() for t in before))
    o2, lse2 = fa.forward_kv4(q, other, lens, table, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(cache.weights, other.weights)
    assert np.isclose(float((cache.weights - before[4]).sum()), B * Hkv * G * n_q, rtol=1e-3)
    assert fa.fa_get_device_status(0) == 0
