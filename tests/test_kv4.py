"""The 4-bit KV cache: append, read, attention, eviction, and key weights.

Everything that is whole numbers or moved bytes is compared exactly with the
fp64 reference (oracle/kv4.py).  Computed outputs are compared within bounds
made of the formats, per output:

S    a score is a sum of d products, exact in what the MMA multiplies, added in fp32 (each of
     the at most d + 4 additions is off by at most 2^-23 of the largest partial sum, which
     sum |q k| scale bounds).  Its product with scale log2 e and the subtraction of the maximum
     round by 2^-24 each.  q goes in as two E4M3 parts, scaled to a maximum of at least 2^7, the second
     16 times larger: their steps are 2^-9 / 16 at the least, so an element is off by at most
     2^-14 of 2^7, 2^-21 of the row's maximum (and exact from 2^-6 on: eight bits in two times four).
     eS = (d + 8) 2^-23 sum |q k| scale + 2^-21 max |q| sum |k| scale.
LSE  its scores' error, and fp32's: eS + 2^-22 (|LSE| + 1).
w    a probability is off by the factor exp(eS + error of LSE) and the exponential's 2^-22:
     w (2 eS + 2^-21 (|LSE| + 2)), a sum of n rows in fp32 adds n 2^-24.
O    the weights' relative error on sum p |v|; what a P in two E4M3 parts may be off by (the kernel's is closer, check_tail holds it to that): the first is off by half a step, at most 2^-4,
     the second by 2^-4 of that, 2^-8 together; the smallest steps, as above, 2^-14 of a scale of 256 that
     stands for at most 2^3 times the row's largest term and four times the largest V scale: 2^-17 times 6
     (a code) times that scale a key, over the sum l; and bf16's rounding of the result (eight significant bits: half a step is 2^-8 of the value).
"""
import numpy as np
import pytest
import torch

import exact_attention_32_gb300 as fa
from oracle import kv4 as ref

gpu = pytest.mark.gpu


def dev(x):
    return torch.as_tensor(np.ascontiguousarray(x)).cuda()


def bf16(x):
    return torch.as_tensor(np.asarray(x, dtype=np.float32)).bfloat16()


def f64(t):
    return t.double().cpu().numpy()


class Pool:
    """A filled cache with the pages of B sequences shuffled in it, unused pages and slots holding rubbish: any code,
    and scale 255 (NaN).  `lens` may be shorter than what is stored."""

    def __init__(self, B, Hkv, d, P, stored, seed, spare=2, gain=1.0):
        rng = np.random.default_rng(seed)
        self.B, self.Hkv, self.d, self.P = B, Hkv, d, P
        stored = np.asarray(stored)
        self.cols = max(1, -(-int(stored.max()) // P)) + 1
        need = [-(-int(n) // P) for n in stored]
        order = rng.permutation(sum(need) + spare)
        self.n_pages = len(order)
        self.table = np.full((B, self.cols), -7, dtype=np.int32)  # entries past the last page are never read
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.n_pages, Hkv, P)
        self.k = rng.integers(0, 256, (*shape, d // 2), dtype=np.uint8)
        self.v = rng.integers(0, 256, (*shape, d // 2), dtype=np.uint8)
        self.ks = np.full((*shape, d // 32), 255, dtype=np.uint8)
        self.vs = np.full(shape, 255, dtype=np.uint8)
        self.w = rng.random(shape, dtype=np.float32)
        for b, n in enumerate(stored):
            if n:
                j = np.arange(n)
                pg, sl = self.table[b, j // P], j % P
                k, ks = ref.quantise(f64(bf16(gain * rng.standard_normal((n, Hkv, d)))), 32)
                v, vs = ref.quantise(f64(bf16(gain * rng.standard_normal((n, Hkv, d)))), d)
                self.k[pg, :, sl], self.ks[pg, :, sl] = k, ks
                self.v[pg, :, sl], self.vs[pg, :, sl] = v, vs[..., 0]

    def cache(self):
        return fa.KV4Cache(dev(self.k), dev(self.v), dev(self.ks), dev(self.vs), dev(self.w))

    def largest_v_scale(self, b, n):
        return ref.SCALES[ref.rows(self.vs, self.table[b], n, self.P)].max() if n else 0.0

    def kv(self, b, n):
        r = lambda t: ref.rows(t, self.table[b], n, self.P)  # noqa: E731
        return ref.values(r(self.k), r(self.ks)), ref.values(r(self.v), r(self.vs)[..., None])


def ok():
    torch.cuda.synchronize()
    assert fa.fa_get_device_status(0) == 0


# ------------------------------------------------------------------- the reference (CPU)

def test_reference_rounds_to_the_nearest_value_of_the_grid():
    rng = np.random.default_rng(0)
    x = f64(bf16(rng.standard_normal((50, 64)) * np.exp(4 * rng.standard_normal((50, 1)))))
    code, s = ref.quantise(x, 32)
    y = ref.values(code, s).reshape(50, 2, 32)
    step = ref.SCALES[s][..., None]
    grid = np.concatenate([-ref.E2M1[::-1], ref.E2M1]) * step[..., None]
    best = np.abs(x.reshape(50, 2, 32)[..., None] - grid).min(-1)
    assert (np.abs(x.reshape(50, 2, 32) - y) == best).all()


def test_reference_attention_is_the_textbook_softmax():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((4, 3, 8)), rng.standard_normal((2, 5, 8)), rng.standard_normal((2, 5, 8))
    r = ref.attention(q, k, v, 0.3, 5)
    e = np.exp(0.3 * k[1, :4] @ q[3, 1])
    assert np.allclose(r["o"][3, 1], e / e.sum() @ v[1, :4], atol=1e-14) and np.isclose(r["lse"][3, 1], np.log(e.sum()))
    assert np.isclose(r["weights"].sum(), 4 * 3) and r["weights"][0, 4] < r["weights"].sum()


def test_reference_eviction_orders_ties_and_nan():
    w = np.array([1.0, 3.0, 3.0, np.nan, 0.0, 3.0, 9.0, 9.0])
    assert ref.evict(w, 8, 5, 2).tolist() == [1, 2, 3, 6, 7]
    assert ref.evict(w, 8, 8, 0).tolist() == list(range(8)) and ref.evict(w, 3, 5, 1).tolist() == [0, 1, 2]


# -------------------------------------------------------------------------- refusals (CPU)

def _struct(**kw):
    f = dict(k=1 << 12, v=1 << 13, k_scale=1 << 14, v_scale=1 << 15, weights=1 << 16, n_pages=8, Hkv=2, page_size=16, d=64)
    f.update(kw)
    return fa.KV4CacheStruct(*[f[n] for n, _ in fa.KV4CacheStruct._fields_])


BAD_CACHES = [(dict(n_pages=0), 1), (dict(n_pages=1 << 31), 1), (dict(Hkv=0), 1), (dict(Hkv=1 << 21), 1),
              (dict(page_size=8), 1), (dict(page_size=48), 1), (dict(page_size=2048), 1), (dict(d=0), 1), (dict(d=96), 2),
              (dict(n_pages=1 << 30, Hkv=1 << 10), 1)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches_are_refused_before_any_device_call(kw, code):
    c, p = _struct(**kw), 1 << 20
    assert fa.fa_kv4_append(c, p, p, None, None, p, p, 1, 1, 1, 0) == code
    assert fa.fa_kv4_read(c, None, p, p, 1, 1, 1, p, p, 0) == code
    assert fa.fa_fwd_kv4(p, c, p, p, p, p, 1, 2, 1, 1, 0.1, 0, p, 1 << 40, 0) == code
    assert fa.fa_kv4_evict(c, p, p, 1, c, p, 1, 1, 1, 0, p, p, 0) == code
    assert fa.fa_kv4_evict(_struct(), p, p, 1, c, p, 1, 1, 1, 0, p, p, 0) == code


def test_bad_arguments_are_refused_before_any_device_call():
    p, c, none = 1 << 20, _struct(), _struct(weights=None)
    INV = 1
    for B, S, pages in [(0, 1, 1), (1, 0, 1), (1, 1, 0), (1 << 40, 1, 1), (1, 1 << 31, 1), (1, 1, 1 << 31)]:
        assert fa.fa_kv4_append(c, p, p, None, None, p, p, B, S, pages, 0) == INV
        assert fa.fa_kv4_read(c, None, p, p, B, pages, S, p, p, 0) == INV
    assert fa.fa_kv4_append(none, p, p, p, None, p, p, 1, 1, 1, 0) == INV  # weights for a cache without
    ws = 1 << 40
    for kw in [dict(B=0), dict(H=0), dict(H=3), dict(n_q=0), dict(n_q=65), dict(H=2 * 512, n_q=3), dict(pages=0),
               dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(acc=2), dict(ws=255)]:
        a = dict(B=1, H=2, n_q=1, pages=1, scale=0.1, acc=0, ws=ws)
        a.update(kw)
        assert fa.fa_fwd_kv4(p, c, p, p, p, p, a["B"], a["H"], a["n_q"], a["pages"], a["scale"], a["acc"], p, a["ws"], 0) == INV
    assert fa.fa_fwd_kv4(p, none, p, p, p, p, 1, 2, 1, 1, 0.1, 1, p, ws, 0) == INV
    for other in [_struct(Hkv=3), _struct(page_size=32), _struct(d=128), none]:
        assert fa.fa_kv4_evict(c, p, p, 1, other, p, 1, 1, 1, 0, p, p, 0) == INV
    for keep, recent in [(0, 0), (17, 0), (4, 5), (4, -1)]:
        assert fa.fa_kv4_evict(c, p, p, 1, c, p, 1, 1, keep, recent, p, p, 0) == INV
    for kw in [dict(H=0), dict(Hkv=0), dict(H=3), dict(N=0), dict(scale=-1.0), dict(causal=2), dict(first=-1), dict(first=8)]:
        a = dict(B=1, H=2, Hkv=2, N=8, d=64, scale=0.1, causal=0, first=0)
        a.update(kw)
        assert fa.fa_key_weights(p, p, p, p, *a.values(), 0) == INV
    assert fa.fa_key_weights(p, p, p, p, 1, 2, 2, 8, 96, 0.1, 0, 0, 0) == 2


def test_capacities_that_pass_31_bits_are_refused():
    c, x = _struct(d=64, Hkv=1, page_size=1024), 1 << 20
    for pages in (1 << 21, (1 << 21) - 1023):
        assert fa.fa_kv4_read(c, 0, x, x, 1, pages, 1, x, x, 0) == 1
    assert fa.fa_fwd_kv4_workspace_bytes(1, 1, 1, 1, 64, (1 << 31) - (1 << 20), 0) > 0
    assert fa.fa_fwd_kv4_workspace_bytes(1, 1, 1, 1, 64, (1 << 31) - (1 << 20) + 1, 0) == -1


def test_workspace_bytes():
    f = fa.fa_fwd_kv4_workspace_bytes
    assert f(1, 8, 2, 1, 96, 64, 0) == -1 and f(1, 7, 2, 1, 64, 64, 0) == -1 and f(1, 8, 2, 0, 64, 64, 0) == -1
    small, long = f(1, 8, 2, 1, 64, 64, 0), f(1, 8, 2, 1, 64, 1 << 17, 0)
    assert 0 < small < long and f(1, 8, 2, 1, 64, 1 << 17, 1) >= long + 8 * (1 << 17) * 4


def test_python_calls_refuse_wrong_tensors():
    c = fa.kv4_cache(2, 1, 16, 64, device="cpu")
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.kv4_read(c, i, i[None], 1)  # not on a CUDA device
    with pytest.raises(ValueError):
        fa.kv4_read(c._replace(v=c.v[:1]), i, i[None], 1)
    with pytest.raises(ValueError):
        fa.kv4_read(c._replace(k=c.k[0]), i, i[None], 1)
    with pytest.raises(fa.FAError):
        fa.kv4_cache(2, 1, 16, 96, device="cpu")
    with pytest.raises(ValueError):
        fa.key_weights(torch.zeros(1, 3, 8, 64).bfloat16(), torch.zeros(1, 2, 8, 64).bfloat16(), torch.zeros(1, 3, 8))


def test_python_calls_refuse_what_is_no_tensor_or_cache():
    c = fa.kv4_cache(2, 1, 16, 64, device="cpu")
    i = torch.zeros(1, dtype=torch.int32)
    for cache in (None, tuple(c)[:4], (1, 2, 3, 4, 5), c._replace(k=[0]), c._replace(k=torch.zeros(2, 1, 16, 32, dtype=torch.uint8).to_sparse())):
        with pytest.raises(ValueError):
            fa.kv4_read(cache, i, i[None], 1)
    with pytest.raises(ValueError):
        fa.key_weights(None, None, None)
    with pytest.raises(TypeError):
        fa.kv4_read(c, i)


@gpu
def test_python_calls_refuse_wrong_gpu_tensors():
    c = fa.kv4_cache(4, 2, 16, 64)
    i, x = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    t = i[None]
    for bad in (x.float(), x[:, :1], x[..., :32], x.cpu(), x.expand(2, 2, 1, 64), x.transpose(1, 2), None):
        with pytest.raises(ValueError):
            fa.kv4_append(c, x, bad, i, t)
    for lens in (i.long(), i[None], i.cpu(), torch.zeros(2, dtype=torch.int32, device="cuda"), 0):
        with pytest.raises(ValueError):
            fa.kv4_append(c, x, x, lens, t)
    with pytest.raises(ValueError):
        fa.kv4_read(c._replace(v=c.v.cpu()), i, t, 1)
    with pytest.raises(ValueError):
        fa.kv4_read(c, i, t, 0)
    with pytest.raises(TypeError):
        fa.kv4_read(c, i, t, 1.5)
    with pytest.raises(ValueError):
        fa.forward_kv4(x[:, :1].contiguous(), c, i, t)  # 1 head over 2 key heads
    with pytest.raises(TypeError):
        fa.forward_kv4(x, c, i, t, scale="1")
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(fa.FAError):
            fa.forward_kv4(x, c, i, t, scale=scale)
    with pytest.raises(ValueError):
        fa.forward_kv4(x, c, i, t, workspace=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        fa.forward_kv4(x, c._replace(weights=None), i, t, accumulate=True)
    with pytest.raises(ValueError):
        fa.kv4_evict(c, i, t, fa.kv4_cache(4, 2, 32, 64), t, 1)
    with pytest.raises(ValueError):
        fa.kv4_evict(c, i, t, c, t, 17)
    ok()


# ------------------------------------------------------------------------------- append, read

SPECIAL = np.array([0.0, -0.0, 1e-30, 2.0 ** -18 * 6, 2.0 ** -17 * 5, 3e-4, 0.1, 1.0, 5.0, 6.0, 448.0, 61440.0, 65000.0, 3e38])


def _hard_rows(rng, n, d):
    """Rows whose blocks have every size, values in the middle of two codes, zeros, and non-finite ones."""
    x = rng.standard_normal((n, d)) * np.exp(5 * rng.standard_normal((n, 1)))
    x[0] = 0
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for i in range(1, min(n, 12)):  # middles times a scale of four significant bits: exact in bf16
        s = (8 + rng.integers(0, 8)) / 8 * 2.0 ** rng.integers(-14, 9)
        x[i] = np.tile(mid, d // 8) * s * np.where(rng.random(d) < 0.5, -1, 1)
    for i in range(12, min(n, 12 + len(SPECIAL))):
        x[i] = SPECIAL[i - 12] * np.where(rng.random(d) < 0.5, -1, rng.random(d))
    if n > 30:
        x[27, 3], x[28, d - 1], x[29, 5] = np.nan, np.inf, -np.inf
    return x


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hkv,S,P", [(1, 1, 1, 16), (3, 2, 37, 16), (2, 5, 130, 64), (1, 3, 300, 1024)])
def test_append_writes_the_reference_codes_and_nothing_else(B, Hkv, S, P, d):
    rng = np.random.default_rng(B * 1000 + S + d)
    k = bf16(np.stack([_hard_rows(rng, Hkv * S, d) for _ in range(B)]).reshape(B, Hkv, S, d))
    v = bf16(np.stack([_hard_rows(rng, Hkv * S, d) for _ in range(B)]).reshape(B, Hkv, S, d))
    n_new = rng.integers(0, S + 1, B)
    n_new[0] = S
    lens = n_new + rng.integers(0, 50, B)
    pool = Pool(B, Hkv, d, P, lens, seed=S)
    w = rng.random((B, Hkv, S), dtype=np.float32)
    for given in (True, False):
        c = pool.cache()
        fa.kv4_append(c, k.cuda(), v.cuda(), dev(lens.astype(np.int32)), dev(pool.table), n_new=dev(n_new.astype(np.int32)),
                      weights=dev(w) if given else None)
        ok()
        want = [pool.k.copy(), pool.v.copy(), pool.ks.copy(), pool.vs.copy(), pool.w.copy()]
        for b in range(B):
            n = n_new[b]
            j = np.arange(lens[b] - n, lens[b])
            pg, sl = pool.table[b, j // P], j % P
            kc, ks = ref.quantise(f64(k[b, :, :n]), 32)
            vc, vs = ref.quantise(f64(v[b, :, :n]), d)
            for t, x in zip(want, (kc, vc, ks, vs[..., 0], w[b, :, :n] if given else 0 * w[b, :, :n])):
                t[pg, :, sl] = np.moveaxis(x, 0, 1)
        for got, t in zip(c, want):
            assert torch.equal(got.cpu(), torch.as_tensor(t))


@gpu
def test_append_without_counts_or_weights():
    B, Hkv, S, d, P = 2, 2, 3, 64, 16
    pool = Pool(B, Hkv, d, P, [3, 20], seed=5)
    x = bf16(np.random.default_rng(6).standard_normal((B, Hkv, S, d)))
    c = pool.cache()._replace(weights=None)
    fa.kv4_append(c, x.cuda(), x.cuda(), dev(np.array([3, 20], np.int32)), dev(pool.table))
    ok()
    kc, _ = ref.quantise(f64(x), 32)
    got = c.k.cpu().numpy()
    for b, at in ((0, 0), (1, 17)):
        for i in range(S):
            j = at + i
            assert (got[pool.table[b, j // P], :, j % P] == kc[b, :, i]).all()


@gpu
@pytest.mark.parametrize("S,over", [(1, 1), (8, 3), (8, 8), (8, 100), (300, 290), (4, 2 ** 31 - 1 - 48), (4, -48 - 3), (4, -(2 ** 31) - 48)])
def test_append_past_the_table_drops_what_has_no_place(S, over):
    # the length after the append is `over` tokens past the table's 48 (or before 0): tokens with a place go there, the others
    # nowhere, and no row that is stored changes
    d, P, cap = 64, 16, 48
    pool = Pool(2, 2, d, P, [cap, 20], seed=S + 1000)
    pool.table = np.ascontiguousarray(pool.table[:, :cap // P])
    x = bf16(np.random.default_rng(S).standard_normal((2, 2, S, d)))
    n = np.array([S, 0], np.int32)
    c = pool.cache()
    fa.kv4_append(c, x.cuda(), x.cuda(), dev(np.array([cap + over, 20], np.int32)), dev(pool.table), n_new=dev(n))
    torch.cuda.synchronize()
    assert fa.fa_get_device_status(0) == 8 and fa.fa_get_device_status(0) == 0
    want = [pool.k.copy(), pool.v.copy(), pool.ks.copy(), pool.vs.copy(), pool.w.copy()]
    at = cap + over - S + np.arange(S, dtype=np.int64)
    i = np.flatnonzero((at >= 0) & (at < cap))
    pg, sl = pool.table[0, at[i] // P], at[i] % P
    (kc, ks), (vc, vs) = ref.quantise(f64(x[0]), 32), ref.quantise(f64(x[0]), d)
    for t, y in zip(want, (kc, vc, ks, vs[..., 0], np.zeros((2, S)))):
        t[pg, :, sl] = np.moveaxis(y[:, i], 0, 1)
    for got, t in zip(c, want):
        assert torch.equal(got.cpu(), torch.as_tensor(t))


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [16, 128])
def test_read_gives_the_stored_values_and_zeros_behind_them(P, d):
    lens = np.array([0, 1, 16, 77, 200], np.int32)
    pool = Pool(5, 3, d, P, lens, seed=d + P)
    first = np.array([0, 0, 5, -3, 190], np.int32)
    k, v = fa.kv4_read(pool.cache(), dev(lens), dev(pool.table), 33, first=dev(first))
    ok()
    for b in range(5):
        kk, vv = pool.kv(b, lens[b])
        for i in range(33):
            j = first[b] + i
            for got, x in ((k, kk), (v, vv)):
                assert (f64(got[b, :, i]) == (x[:, j] if 0 <= j < lens[b] else 0)).all()
    k0, _ = fa.kv4_read(pool.cache(), dev(lens), dev(pool.table), 300)
    assert torch.equal(k0[4, :, 190:200], k[4, :, :10]) and (k0[4, :, 200:] == 0).all()


# ----------------------------------------------------------------------------------- attention

def check_attention(pool, q, lens, scale, o, lse, w_before=None, w_after=None, gone=()):
    B, H, n_q, d = q.shape
    o, lse, qd = f64(o), f64(lse), f64(q)
    want_w = None if w_before is None else w_before.astype(np.float64)
    tol_w = None if w_before is None else np.zeros_like(want_w)
    for b in range(B):
        n = int(lens[b])
        k, v = pool.kv(b, n)
        r = ref.attention(qd[b], k, v, scale, n)
        eS = (d + 8) * 2.0 ** -23 * r["reach"] + 2.0 ** -21 * r["top_q"]
        none = r["lse"] == -np.inf
        assert (lse[b][none] == -np.inf).all() and (o[b][none] == 0).all()
        live = ~none
        top = np.where(live, np.abs(r["lse"]), 0)
        assert (np.abs(lse[b][live] - r["lse"][live]) <= (eS + 2.0 ** -22 * (top + 1))[live]).all()
        rel = 2 * eS + 2.0 ** -21 * (top + 2)
        tiny = n * 2.0 ** -17 * 6 * pool.largest_v_scale(b, n) / r["total"]
        tol = (rel + 2.0 ** -8)[..., None] * r["spread"] + tiny[..., None] + 2.0 ** -8 * np.abs(r["o"])
        err = np.abs(o[b] - r["o"])
        assert (err <= tol).all(), (b, (err / np.maximum(tol, 1e-300)).max())
        if want_w is not None and n:
            j = np.arange(n)
            pg, sl = pool.table[b, j // pool.P], j % pool.P
            want_w[pg, :, sl] += r["weights"].T
            G = H // pool.Hkv
            worst = rel.reshape(pool.Hkv, G * n_q).max(-1)
            tol_w[pg, :, sl] = (r["weights"] * worst[:, None]).T + 2.0 ** -24 * (G * n_q + 2) * want_w[pg, :, sl]
    if want_w is not None:
        assert (np.abs(w_after - want_w) <= tol_w).all()


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv,G,n_q", [(1, 1, 1), (2, 4, 1), (1, 8, 1), (3, 7, 1), (2, 1, 5), (1, 3, 4), (2, 16, 1),
                                       (1, 8, 3), (1, 16, 8), (2, 2, 64)])
def test_attention_over_short_and_odd_lengths(Hkv, G, n_q, d):
    # 0 and 1 token; fewer tokens than queries (rows that admit nothing); tile and page borders and beside them
    lens = np.array([0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255, 256, 257, 300], np.int32)
    pool = Pool(len(lens), Hkv, d, 16, lens, seed=Hkv * 100 + G * 10 + n_q)
    q = bf16(np.random.default_rng(G).standard_normal((len(lens), Hkv * G, n_q, d))).cuda()
    scale = fa.default_scale(d)
    c = pool.cache()
    o, lse = fa.forward_kv4(q, c, dev(lens), dev(pool.table), accumulate=True)
    o2, lse2 = fa.forward_kv4(q, c, dev(lens), dev(pool.table))
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_attention(pool, q, lens, scale, o, lse, pool.w, f64(c.weights))


@gpu
@pytest.mark.parametrize("d,P,Hkv,G,n_q", [(128, 64, 2, 4, 1), (64, 32, 1, 8, 2), (128, 1024, 1, 1, 1), (128, 16, 1, 12, 2)])
def test_attention_over_long_ragged_lengths(d, P, Hkv, G, n_q):
    # several chunks, some sequences far shorter than the table's columns
    lens = np.array([9000, 4097, 1, 700], np.int32)
    pool = Pool(4, Hkv, d, P, lens, seed=d + P)
    q = bf16(3 * np.random.default_rng(G).standard_normal((4, Hkv * G, n_q, d))).cuda()
    c = pool.cache()
    o, lse = fa.forward_kv4(q, c, dev(lens), dev(pool.table), scale=0.11, accumulate=True)
    ok()
    check_attention(pool, q, lens, float(np.float32(0.11)), o, lse, pool.w, f64(c.weights))


@gpu
@pytest.mark.parametrize("d,P,B,n_q,stored", [(64, 16, 700, 1, 80), (128, 16, 1300, 2, 40), (128, 32, 450, 1, 900), (64, 64, 400, 3, 1500)])
def test_attention_over_many_sequences(d, P, B, n_q, stored):
    # more sequences than a CTA has threads, most of them shorter than a tile, among them empty ones
    rng = np.random.default_rng(B)
    lens = rng.integers(0, stored // 8, B).astype(np.int32)
    lens[::37], lens[5], lens[B - 1] = 0, stored, stored - 1
    pool = Pool(B, 1, d, P, lens, seed=B)
    q = bf16(rng.standard_normal((B, 3, n_q, d))).cuda()
    c = pool.cache()
    o, lse = fa.forward_kv4(q, c, dev(lens), dev(pool.table), accumulate=True)
    ok()
    check_attention(pool, q, lens, fa.default_scale(d), o, lse, pool.w, f64(c.weights))


@gpu
@pytest.mark.parametrize("d,P,Hkv,G,n_q,lens", [(128, 1024, 1, 2, 1, [1024, 0, 1023]), (64, 16, 2, 4, 2, [640, 640, 1]),
                                                (64, 1024, 1, 1, 3, [4096, 4095, 2]), (128, 16, 1, 16, 64, [640, 63, 64]),
                                                (64, 16, 1, 1024, 1, [700, 32, 5]), (128, 16, 2, 2, 1, [640, 333, 1]), (64, 32, 1, 20, 1, [640, 333, 1]), (128, 128, 1, 33, 1, [1280, 129, 1])])
def test_attention_over_full_tables_and_many_rows(d, P, Hkv, G, n_q, lens):
    # sequences as long as the table allows, and up to 1024 rows a key head
    lens = np.array(lens, np.int32)
    pool = Pool(len(lens), Hkv, d, P, lens, seed=P + G)
    pool.table = np.ascontiguousarray(pool.table[:, :-(-int(lens.max()) // P)])
    q = bf16(np.random.default_rng(G).standard_normal((len(lens), Hkv * G, n_q, d))).cuda()
    c = pool.cache()
    o, lse = fa.forward_kv4(q, c, dev(lens), dev(pool.table), accumulate=True)
    ok()
    check_attention(pool, q, lens, fa.default_scale(d), o, lse, pool.w, f64(c.weights))


@gpu
@pytest.mark.parametrize("gain", [1e-4, 1e3])
@pytest.mark.parametrize("q_gain", [1e-20, 1e-3, 40.0])
def test_attention_over_small_and_large_values(gain, q_gain):
    lens = np.array([100, 513], np.int32)
    pool = Pool(2, 1, 128, 32, lens, seed=3, gain=gain)
    q = bf16(q_gain / gain * np.random.default_rng(2).standard_normal((2, 4, 1, 128))).cuda()
    o, lse = fa.forward_kv4(q, pool.cache(), dev(lens), dev(pool.table))
    ok()
    check_attention(pool, q, lens, fa.default_scale(128), o, lse)


def _put(pool, b, j, k=None, v=None):
    """Token j of sequence b becomes the rows k, v (each [Hkv, d], or None to leave what is there)."""
    at = pool.table[b, j // pool.P], slice(None), j % pool.P
    if k is not None:
        pool.k[at], pool.ks[at] = ref.quantise(f64(bf16(k)), 32)
    if v is not None:
        code, s = ref.quantise(f64(bf16(v)), pool.d)
        pool.v[at], pool.vs[at] = code, s[..., 0]


def check_tail(pool, q, lens, scale, copies):
    """Attention over the pool's sequences, each `copies` times in the batch (many copies make long shares, cut in other places in
    each).  O within 2^-10 of sum p |v| and bf16's rounding (2^-8 of the value), beside the scores' error (as above): whatever a
    row's largest terms are, the small ones count, and nothing grows with the number of keys.  p s (s: V's scale) is rounded to a
    half: 2^-11 of itself down to 2^-24 of the row's largest one, which none of the keys here that matter lies below; each of the sums
    over n / 32 products is off by at most 2^-23 of it: 2^-14 at 16384 keys."""
    B = len(lens)
    o, lse = fa.forward_kv4(q.repeat(copies, 1, 1, 1), pool.cache(), dev(np.tile(lens, copies)), dev(np.tile(pool.table, (copies, 1))))
    ok()
    o, lse = f64(o).reshape(copies, *q.shape), f64(lse).reshape(copies, *q.shape[:-1])
    for b in range(B):
        n = int(lens[b])
        r = ref.attention(f64(q[b]), *pool.kv(b, n), scale, n)
        eS = (pool.d + 8) * 2.0 ** -23 * r["reach"] + 2.0 ** -21 * r["top_q"]
        assert (np.abs(lse[:, b] - r["lse"]) <= eS + 2.0 ** -22 * (np.abs(r["lse"]) + 1)).all()
        rel = 2 * eS + 2.0 ** -21 * (np.abs(r["lse"]) + 2)
        err, tol = np.abs(o[:, b] - r["o"]), (rel + 2.0 ** -10)[..., None] * r["spread"] + 2.0 ** -8 * np.abs(r["o"])
        assert (err <= tol).all(), (b, (err / tol).max(), np.sqrt((err[0] ** 2).sum() / (r["o"] ** 2).sum()))


@gpu
@pytest.mark.parametrize("Hkv,G,n_q,d", [(2, 1, 1, 64), (1, 4, 1, 128), (1, 12, 1, 64), (1, 8, 2, 128), (1, 32, 1, 64), (1, 8, 5, 128)])
@pytest.mark.parametrize("n,at,copies", [(300, 0, 1), (2048, 0, 200), (2048, 1000, 1), (16384, 0, 1), (16384, 5000, 150)])
def test_attention_behind_a_heavy_key_keeps_the_others(n, at, copies, Hkv, G, n_q, d):
    # a key 8, 11 or 14 nats above the others' mean whose V is small (an attention sink), first or in the middle
    lens = np.array([n, n - 7, n // 2 + at], np.int32)
    pool = Pool(3, Hkv, d, 64, lens, seed=n + at + G)
    rng = np.random.default_rng(G + d)
    scale = fa.default_scale(d)
    q = rng.standard_normal((3, Hkv * G, n_q, d))
    q[..., 0] = 16.0  # channel 0 is the heavy key's alone
    pool.k[..., 0] &= 0xF0
    for b, nats in enumerate((8.0, 11.0, 14.0)):
        k, v = np.zeros((Hkv, d)), rng.standard_normal((Hkv, d)) / 64
        k[:, 0] = nats / (scale * 16.0)
        _put(pool, b, at, k, v)
    check_tail(pool, bf16(q).cuda(), lens, scale, copies)


@gpu
@pytest.mark.parametrize("Hkv,G,n_q,d", [(2, 4, 1, 64), (1, 4, 2, 128), (1, 12, 1, 128), (1, 16, 2, 64)])
@pytest.mark.parametrize("gain", [64.0, 300.0, 4096.0])
def test_a_large_value_of_next_to_no_weight_leaves_the_others_alone(gain, Hkv, G, n_q, d):
    # a V row `gain` times the others' at a key far below them; and one that only the last query admits
    lens = np.array([8192, 8192], np.int32)
    pool = Pool(2, Hkv, d, 64, lens, seed=int(gain) + G)
    rng = np.random.default_rng(G + d)
    scale = fa.default_scale(d)
    q = rng.standard_normal((2, Hkv * G, n_q, d))
    q[..., 0] = 16.0
    pool.k[..., 0] &= 0xF0
    for b, j in ((0, 0), (1, 8191)):
        k = np.zeros((Hkv, d))
        k[:, 0] = -20.0 / (scale * 16.0)
        _put(pool, b, j, k, gain * rng.standard_normal((Hkv, d)))
    check_tail(pool, bf16(q).cuda(), lens, scale, 250)


@gpu
@pytest.mark.parametrize("d,G", [(64, 8), (128, 8), (128, 16), (64, 32)])
def test_heavy_keys_without_values_and_rising_scores(d, G):
    # V scale 0 at the heaviest keys (their terms vanish, the others' remain), scores that rise and fall over the sequence by 25 nats, V
    # that falls and rises against them
    n = 6000
    lens = np.array([n, n], np.int32)
    pool = Pool(2, 1, d, 128, lens, seed=d + G)
    rng = np.random.default_rng(G)
    scale = fa.default_scale(d)
    q = rng.standard_normal((2, G, 1, d))
    q[..., 0] = 16.0
    for b in range(2):
        for j in range(n):
            nats = (j * 25 / n) if b else 25 - j * 25 / n
            k, v = 0.5 * rng.standard_normal((1, d)), rng.standard_normal((1, d)) * np.exp(0.8 * (12 - nats))
            k[:, 0] = nats / (scale * 16.0)
            _put(pool, b, j, k, 0 * v if j % 97 == 5 else v)
        k[:, 0] = 30.0 / (scale * 16.0)
        _put(pool, b, 3000, k, np.zeros((1, d)))
    for copies in (1, 250):
        check_tail(pool, bf16(q).cuda(), lens, scale, copies)


@gpu
def test_a_stored_nan_reaches_the_rows_that_admit_it_and_no_other():
    lens = np.array([40, 40], np.int32)
    pool = Pool(2, 1, 64, 16, lens, seed=11)
    pool.vs[pool.table[0, 39 // 16], 0, 39 % 16] = 255  # the last token: only the last query admits it
    pool.ks[pool.table[1, 38 // 16], 0, 38 % 16, 1] = 255
    q = bf16(np.random.default_rng(3).standard_normal((2, 2, 3, 64))).cuda()
    o, lse = (f64(x) for x in fa.forward_kv4(q, pool.cache(), dev(lens), dev(pool.table)))
    ok()
    assert np.isfinite(o[0, :, :2]).all() and np.isnan(o[0, :, 2]).all() and np.isfinite(lse[0]).all()
    assert np.isfinite(o[1, :, 0]).all() and np.isnan(o[1, :, 1:]).all() and np.isnan(lse[1, :, 1:]).all()


@gpu
@pytest.mark.parametrize("d,G,n", [(64, 1, 40), (128, 2, 70), (64, 4, 300), (128, 8, 3000), (64, 16, 2000)])
def test_a_row_of_nan_weighs_no_key_that_it_does_not_admit(d, G, n):
    # three new tokens: the first of them has a NaN in q (every head's).  The two newest keys are not among those that it admits: their
    # weights are the other queries'
    lens = np.array([n, 2], np.int32)  # (of the second sequence's rows the first admits nothing at all)
    pool = Pool(2, 1, d, 16, lens, seed=n)
    q = np.random.default_rng(n).standard_normal((2, G, 3, d))
    q[:, :, 0, 7] = np.nan
    c = pool.cache()
    o, lse = fa.forward_kv4(bf16(q).cuda(), c, dev(lens), dev(pool.table), accumulate=True)
    ok()
    got = f64(c.weights)
    q[:, :, 0] = 0
    for b in range(2):
        j = np.arange(int(lens[b]))
        added = got[pool.table[b, j // 16], 0, j % 16] - pool.w[pool.table[b, j // 16], 0, j % 16]
        r = ref.attention(f64(bf16(q[b])), *pool.kv(b, len(j)), fa.default_scale(d), len(j))
        first = max(0, len(j) - 2)
        assert np.isnan(added[:first]).all() and np.isnan(f64(o[b, :, 0])).all() == (first > 0)
        assert np.abs(added[first:] - r["weights"][0, first:]).max() <= 1e-4 * G and np.isfinite(f64(o[b, :, 1:])).all()


@gpu
def test_bad_pages_and_lengths_are_left_out_and_reported():
    # the kernels check the table and the lengths themselves: nothing outside the pool is read or written
    lens = np.array([100, 60], np.int32)
    pool = Pool(2, 2, 64, 16, lens, seed=21)
    table = pool.table.copy()
    table[0, 2] = pool.n_pages
    q = bf16(np.random.default_rng(4).standard_normal((2, 4, 1, 64))).cuda()
    c = pool.cache()
    o, lse = fa.forward_kv4(q, c, dev(lens), dev(table), accumulate=True)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status(0) == 8 and fa.fa_get_device_status(0) == 0
    k, v = pool.kv(0, 100)
    left = np.r_[0:32, 48:100]
    r = ref.attention(f64(q[0]), k[:, left], v[:, left], fa.default_scale(64), 84)
    assert np.abs(f64(o[0]) - r["o"]).max() < 2.0 ** -8 * np.abs(r["o"]).max() and np.abs(f64(lse[0]) - r["lse"]).max() < 1e-4
    check_attention_one = ref.attention(f64(q[1]), *pool.kv(1, 60), fa.default_scale(64), 60)
    assert np.abs(f64(o[1]) - check_attention_one["o"]).max() < 2.0 ** -8 * np.abs(check_attention_one["o"]).max()
    # a length past the table's columns, a negative one, a negative position
    cols = pool.cols
    o, lse = fa.forward_kv4(q, c, dev(np.array([-5, 60], np.int32)), dev(pool.table))
    torch.cuda.synchronize()
    assert fa.fa_get_device_status(0) == 8 and (lse[0] == float("-inf")).all() and (o[0] == 0).all()
    full = np.abs(table) % pool.n_pages
    k1, _ = fa.kv4_read(c, dev(np.array([10 ** 6, 60], np.int32)), dev(full.astype(np.int32)), 16 * cols + 5)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status(0) == 8 and (k1[0, :, 16 * cols:] == 0).all()
    before = [t.clone() for t in c]
    x = bf16(np.ones((2, 2, 4, 64))).cuda()
    fa.kv4_append(c, x, x, dev(np.array([0, 0], np.int32)), dev(pool.table))
    torch.cuda.synchronize()
    assert fa.fa_get_device_status(0) == 8 and all(torch.equal(a, b) for a, b in zip(before, c))


@gpu
def test_workspace_is_all_that_is_used_and_small_ones_are_refused():
    lens = np.array([1000], np.int32)
    pool = Pool(1, 1, 64, 16, lens, seed=31)
    q = bf16(np.random.default_rng(5).standard_normal((1, 4, 2, 64))).cuda()
    need = fa.fa_fwd_kv4_workspace_bytes(1, 4, 1, 2, 64, pool.cols * 16, True)
    ws = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    c = pool.cache()
    o, lse = fa.forward_kv4(q, c, dev(lens), dev(pool.table), accumulate=True, workspace=ws[:need])
    o2, lse2 = fa.forward_kv4(q, pool.cache(), dev(lens), dev(pool.table), accumulate=True)
    ok()
    assert (ws[need:] == 171).all() and torch.equal(o, o2) and torch.equal(lse, lse2)
    with pytest.raises(fa.FAError):
        fa.forward_kv4(q, c, dev(lens), dev(pool.table), accumulate=True, workspace=ws[:need - 1])


@gpu
def test_overlapping_and_misplaced_pointers_are_refused():
    lens, pool = np.array([20], np.int32), Pool(1, 1, 64, 16, [20], seed=41)
    c, p = pool.cache(), dev(pool.table)
    n = dev(lens)
    s = fa.KV4CacheStruct(*(t.data_ptr() for t in c), pool.n_pages, 1, 16, 64)
    q = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    ws, lse = torch.empty(1 << 20, dtype=torch.uint8, device="cuda"), torch.zeros(1, device="cuda")
    call = lambda o, l, w: fa.fa_fwd_kv4(q.data_ptr(), s, n.data_ptr(), p.data_ptr(), o, l, 1, 1, 1, p.shape[1], 0.1,  # noqa: E731
                                         0, w, ws.numel(), 0)
    assert call(c.k.data_ptr(), lse.data_ptr(), ws.data_ptr()) == 1
    assert call(q.data_ptr(), lse.data_ptr(), ws.data_ptr()) == 1
    assert call(ws.data_ptr(), lse.data_ptr(), ws.data_ptr()) == 1
    assert call(lse.data_ptr() + 2, lse.data_ptr(), ws.data_ptr()) == 1
    host = torch.zeros(64, dtype=torch.bfloat16)
    assert call(host.data_ptr(), lse.data_ptr(), ws.data_ptr()) == 1
    assert fa.fa_kv4_append(s, c.k.data_ptr(), q.data_ptr(), None, None, n.data_ptr(), p.data_ptr(), 1, 1, p.shape[1], 0) == 1
    assert fa.fa_kv4_read(s, None, n.data_ptr(), p.data_ptr(), 1, p.shape[1], 1, c.v.data_ptr(), q.data_ptr(), 0) == 1
    assert fa.fa_kv4_evict(s, n.data_ptr(), p.data_ptr(), p.shape[1], s, p.data_ptr(), p.shape[1], 1, 4, 0,
                           c.weights.data_ptr(), lse.data_ptr(), 0) == 1
    ok()


# ------------------------------------------------------------------------------------ eviction

def check_eviction(pool, w, lens, keep, recent, same_pool, seed=0):
    B, Hkv, P, d = pool.B, pool.Hkv, pool.P, pool.d
    rng = np.random.default_rng(seed)
    cols = -(-keep // P)
    src = pool.cache()._replace(weights=dev(w))
    if same_pool:  # fresh pages behind the old ones
        grow = lambda t: torch.cat([t, t[:1].expand(B * cols, *t.shape[1:])]).contiguous()  # noqa: E731
        src = to = fa.KV4Cache(*(grow(t) for t in src))
        to_table = (pool.n_pages + rng.permutation(B * cols)).reshape(B, cols).astype(np.int32)
    else:
        to = fa.kv4_cache(B * cols + 1, Hkv, P, d)
        to_table = rng.permutation(B * cols + 1)[:B * cols].reshape(B, cols).astype(np.int32)
    before = [t.cpu().numpy().copy() for t in to]
    kept, now = fa.kv4_evict(src, dev(lens), dev(pool.table), to, dev(to_table), keep, recent=recent)
    ok()
    assert (now.cpu().numpy() == np.minimum(lens, keep)).all()
    kept = kept.cpu().numpy()
    for b in range(B):
        n, m = int(lens[b]), min(int(lens[b]), keep)
        for h in range(Hkv):
            at = ref.evict(ref.rows(w, pool.table[b], n, P)[h] if n else np.zeros(0), n, keep, recent)
            assert (kept[b, h, :m] == at).all() and (kept[b, h, m:] == -1).all()
            i = np.arange(m)
            for t, x in zip(before, (pool.k, pool.v, pool.ks, pool.vs, w)):
                t[to_table[b, i // P], h, i % P] = x[pool.table[b, at // P], h, at % P]
    for got, t in zip(to, before):
        assert np.array_equal(got.cpu().numpy(), t, equal_nan=True)  # the rest of the pages is as it was


@gpu
@pytest.mark.parametrize("same_pool", [False, True])
@pytest.mark.parametrize("d,P,keep,recent", [(64, 16, 1, 0), (64, 16, 1, 1), (128, 16, 40, 8), (64, 64, 100, 100), (128, 32, 200, 0),
                                             (128, 16, 3000, 100)])
def test_eviction_keeps_the_heaviest_and_the_latest(d, P, keep, recent, same_pool):
    lens = np.array([0, 1, 39, 40, 41, 130, 1024, 2500], np.int32)
    pool = Pool(len(lens), 2, d, P, lens, seed=keep + recent)
    rng = np.random.default_rng(keep)
    w = np.exp(2 * rng.standard_normal(pool.w.shape)).astype(np.float32)
    w[rng.random(w.shape) < 0.3] = 0  # ties
    check_eviction(pool, w, lens, keep, recent, same_pool)


@gpu
@pytest.mark.parametrize("kind", ["equal", "signed", "nonfinite", "neighbours"])
def test_eviction_orders_every_float(kind):
    lens = np.array([1500, 333], np.int32)
    pool = Pool(2, 3, 64, 16, lens, seed=7)
    rng = np.random.default_rng(8)
    w = rng.standard_normal(pool.w.shape).astype(np.float32)
    if kind == "equal":
        w[:] = 1.5
    elif kind == "signed":
        w[rng.random(w.shape) < 0.2], w[rng.random(w.shape) < 0.2] = 0.0, -0.0
    elif kind == "nonfinite":
        w[rng.random(w.shape) < 0.1], w[rng.random(w.shape) < 0.1], w[rng.random(w.shape) < 0.1] = np.nan, np.inf, -np.inf
    else:
        w[:] = np.float32(1) + rng.integers(0, 4, w.shape) * np.float32(2.0 ** -23)
    check_eviction(pool, w, lens, 200, 17, False)


@gpu
@pytest.mark.parametrize("n", [16384, 60000, 70001])
def test_eviction_from_long_sequences(n):
    lens = np.array([n, n // 2], np.int32)
    pool = Pool(2, 1, 64, 128, lens, seed=9)
    w = np.exp(np.random.default_rng(10).standard_normal(pool.w.shape)).astype(np.float32)
    check_eviction(pool, w, lens, n // 3, 512, False)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,keep,recent", [([70, 100], 128, 5), ([70, 100], 60, 40), ([100, 100], 1, 1)])
def test_eviction_from_a_bad_page_leaves_rows_of_zeros(lens, keep, recent, d):
    # sequence 0's page 3 and sequence 1's last page are no pages of the pool: what is kept of them is zeros without weight, not what
    # lay in the new pages, and everything else is as without the fault
    lens, P = np.array(lens, np.int32), 16
    pool = Pool(2, 2, d, P, lens, seed=keep, spare=8)
    table = pool.table.copy()
    table[0, 3], table[1, (lens[1] - 1) // P] = pool.n_pages, -1
    to = fa.KV4Cache(*(torch.randint(1, 200, t.shape, device="cuda").to(t.dtype) for t in pool.cache()))
    cols = -(-keep // P)
    to_table = np.arange(2 * cols, dtype=np.int32).reshape(2, cols)
    want = [t.cpu().numpy().copy() for t in to]
    kept, now = fa.kv4_evict(pool.cache(), dev(lens), dev(table), to, dev(to_table), keep, recent=recent)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status(0) == 8 and fa.fa_get_device_status(0) == 0
    kept = kept.cpu().numpy()
    met = 0
    for b in range(2):
        m = min(int(lens[b]), keep)
        assert int(now[b]) == m
        for h in range(2):
            assert (np.diff(kept[b, h, :m]) > 0).all()
            for i, j in enumerate(kept[b, h, :m]):
                src, at = table[b, j // P], (to_table[b, i // P], h, i % P)
                bad = not 0 <= src < pool.n_pages
                met += bad
                for t, x in zip(want, (pool.k, pool.v, pool.ks, pool.vs, pool.w)):
                    t[at] = 0 if bad else x[src, h, j % P]
    assert met
    for got, t in zip(to, want):
        assert np.array_equal(got.cpu().numpy(), t)


# --------------------------------------------------------------------------------- key weights

def _lse(q, k, scale, causal):
    B, H, N, d = q.shape
    s = scale * np.einsum("bhid,bhjd->bhij", q, np.repeat(k, H // k.shape[1], axis=1))
    if causal:
        s = np.where(np.tril(np.ones((N, N), dtype=bool)), s, -np.inf)
    top = s.max(-1)
    return (top + np.log(np.exp(s - top[..., None]).sum(-1))).astype(np.float32)


@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,N,first", [(1, 1, 1, 1, 0), (1, 1, 1, 2, 1), (2, 2, 1, 127, 0), (1, 4, 2, 128, 5), (1, 3, 3, 129, 128),
                                             (2, 8, 1, 255, 0), (1, 2, 2, 256, 200), (1, 7, 1, 257, 0), (1, 2, 1, 511, 300),
                                             (1, 4, 2, 1000, 0), (1, 1, 1, 2049, 2048),
                                             # a few key blocks, shared by the CTAs of a cluster (2 to 8 of them)
                                             (1, 8, 1, 300, 0), (2, 16, 2, 513, 0), (1, 32, 1, 900, 250), (1, 8, 2, 2500, 0)])
def test_key_weights(B, H, Hkv, N, first, d, causal):
    rng = np.random.default_rng(N + H)
    q, k = bf16(rng.standard_normal((B, H, N, d))), bf16(rng.standard_normal((B, Hkv, N, d)))
    scale = fa.default_scale(d)
    lse = _lse(f64(q), f64(k), scale, causal)
    if N > 2:
        lse[0, 0, N // 2] = -np.inf  # a query that admitted no key adds nothing
    w = fa.key_weights(q.cuda(), k.cuda(), dev(lse), causal=causal, first_query=first)
    ok()
    want, reach = ref.key_weights(f64(q), f64(k), lse.astype(np.float64), scale, causal, first)
    top = np.abs(np.where(np.isfinite(lse), lse, 0)).max()
    tol = want * (2 * (d + 8) * 2.0 ** -23 * reach + 2.0 ** -21 * (top + 2)) + 1e-37
    assert w.shape == want.shape and (np.abs(f64(w) - want) <= tol).all()


@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("H,Hkv,N,first", [(2, 1, 200, 0), (2, 2, 700, 300), (16, 1, 515, 129)])
def test_key_weights_of_queries_left_out_may_hold_anything(H, Hkv, N, first, causal):
    # queries before first_query, and those without a key (LSE -inf): NaN, infinities and the largest numbers in them
    g = torch.Generator().manual_seed(N)
    q, k = torch.randn(1, H, N, 64, generator=g).bfloat16(), torch.randn(1, Hkv, N, 64, generator=g).bfloat16()
    lse = dev(_lse(f64(q), f64(k), fa.default_scale(64), causal))
    gone = torch.zeros(N, dtype=torch.bool)
    gone[:first] = True
    gone[first + 3::31] = True
    lse[:, :, torch.arange(first + 3, N, 31)] = -np.inf
    fill = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38]).bfloat16()
    bad = q.clone()
    bad[:, :, gone] = fill[torch.arange(int(gone.sum())) % 4, None]
    w, w2 = (fa.key_weights(x.cuda(), k.cuda(), lse, causal=causal, first_query=first) for x in (q, bad))
    ok()
    assert torch.isfinite(w).all() and torch.equal(w, w2)
    # and a NaN among the others reaches the keys that they admit, no others
    i = int(torch.nonzero(~gone)[len(torch.nonzero(~gone)) // 2])
    q[0, H - 1, i, 5] = float("nan")
    w3 = fa.key_weights(q.cuda(), k.cuda(), lse, causal=causal, first_query=first)
    ok()
    last = i + 1 if causal else N
    assert torch.isnan(w3[0, -1, :last]).all() and torch.equal(w3[0, -1, last:], w[0, -1, last:])
    assert torch.equal(w3[0, :-1], w[0, :-1])


@gpu
@pytest.mark.parametrize("N,real", [(300, 171), (384, 256), (129, 1)])
def test_key_weights_of_a_padded_prompt(N, real):
    # keys and queries past the prompt's end hold NaN, and those queries no LSE: their keys weigh nothing, the others as before
    g = torch.Generator().manual_seed(N)
    q, k = torch.randn(1, 4, N, 128, generator=g).bfloat16(), torch.randn(1, 2, N, 128, generator=g).bfloat16()
    short = dev(_lse(f64(q[:, :, :real]), f64(k[:, :, :real]), fa.default_scale(128), True))
    w = fa.key_weights(q[:, :, :real].contiguous().cuda(), k[:, :, :real].contiguous().cuda(), short, causal=True)
    lse = torch.full((1, 4, N), -np.inf, device="cuda")
    lse[:, :, :real] = short
    q[:, :, real:], k[:, :, real:] = float("nan"), float("nan")
    w2 = fa.key_weights(q.cuda(), k.cuda(), lse, causal=True)
    ok()
    assert (w2[:, :, real:] == 0).all()
    # the same terms, added in blocks that may differ: N roundings of at most 2^-24 of the sum on either side
    assert ((w2[:, :, :real] - w).abs() <= w * 2 * N * 2 * 2.0 ** -24).all()


@gpu
def test_key_weights_sum_to_the_number_of_queries():
    # from the forward's own LSE: the columns of a softmax matrix add up to its rows
    q, k, v = (t.cuda() for t in fa.make_inputs(1, 4, 3000, 128, seed=3))
    _, lse = fa.forward(q, k, v, causal=True)
    w = fa.key_weights(q, k, lse, causal=True)
    half = fa.key_weights(q, k, lse, causal=True, first_query=1500)
    ok()
    # the forward's LSE is within 1e-3 of the truth (its own tests' bound)
    assert (w.double().sum(-1) / 3000 - 1).abs().max() < 1e-3 and (half.double().sum(-1) / 1500 - 1).abs().max() < 1e-3


# --------------------------------------------------------- streams, graphs, all of them together

def _serve(fa_forward, steps, B=2, H=4, Hkv=2, d=64, P=16, N=150, keep=96, recent=16):
    """A prompt, then `steps` tokens with an eviction between: the calls as a program makes them."""
    g = torch.Generator().manual_seed(1)
    randn = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    q, k, v = randn(B, H, N, d), randn(B, Hkv, N, d), randn(B, Hkv, N, d)
    G = H // Hkv
    _, lse = fa.forward(q, k.repeat_interleave(G, 1), v.repeat_interleave(G, 1), causal=True)
    w = fa.key_weights(q, k, lse, causal=True)
    cache = fa.kv4_cache(64, Hkv, P, d)
    order = torch.randperm(64, generator=g).to(torch.int32).cuda()
    table, table2 = order[:B * 16].view(B, 16).contiguous(), order[B * 16:2 * B * 16].view(B, 16).contiguous()
    lens = torch.full((B,), N, dtype=torch.int32, device="cuda")
    fa.kv4_append(cache, k, v, lens, table, weights=w)
    outs, log = [], [(k, v)]
    for s in range(steps):
        if s == steps // 2:
            kept, lens = fa.kv4_evict(cache, lens, table, cache, table2, keep, recent=recent)
            table = table2
            outs.append(kept)
        qn, kn, vn = randn(B, H, 1, d), randn(B, Hkv, 1, d), randn(B, Hkv, 1, d)
        lens = lens + 1
        fa.kv4_append(cache, kn, vn, lens, table)
        o, lse = fa_forward(qn, cache, lens, table)
        outs += [o, lse]
        log.append((qn, kn, vn))
    return outs, log, cache, lens, table, w


@gpu
def test_prompt_decode_evict_decode():
    steps = 8
    outs, log, cache, lens, table, w0 = _serve(lambda *a: fa.forward_kv4(*a, accumulate=True), steps)
    ok()
    (k0, v0), B, H, Hkv, d, G = log[0], 2, 4, 2, 64, 2
    it = iter(outs)
    for b in range(B):
        it = iter(outs)
        K = [ref.values(*ref.quantise(f64(k0[b, h]), 32)) for h in range(Hkv)]
        V = [ref.values(*ref.quantise(f64(v0[b, h]), d)) for h in range(Hkv)]
        W = [f64(w0[b, h]) for h in range(Hkv)]
        for s in range(steps):
            if s == steps // 2:
                kept = next(it)[b].cpu().numpy()
                for h in range(Hkv):
                    # every key kept is at least as heavy as any left out (up to the weights' own rounding)
                    old = np.arange(len(W[h]) - 16)
                    out = np.setdiff1d(old, kept[h])
                    stay = np.intersect1d(old, kept[h])
                    assert len(kept[h]) == 96 and W[h][stay].min() >= W[h][out].max() * (1 - 1e-4)
                    K[h], V[h], W[h] = K[h][kept[h]], V[h][kept[h]], W[h][kept[h]]
            qn, kn, vn = log[1 + s]
            o, lse = next(it), next(it)
            for h in range(Hkv):
                K[h] = np.concatenate([K[h], ref.values(*ref.quantise(f64(kn[b, h]), 32))])
                V[h] = np.concatenate([V[h], ref.values(*ref.quantise(f64(vn[b, h]), d))])
                n = len(K[h])
                r = ref.attention(f64(qn[b, h * G:(h + 1) * G]), K[h][None], V[h][None], fa.default_scale(d), n)
                W[h] = np.concatenate([W[h], [0.0]]) + r["weights"][0]
                assert np.abs(f64(o[b, h * G:(h + 1) * G]) - r["o"]).max() <= 2.0 ** -8 * np.abs(r["o"]).max()
                assert np.abs(f64(lse[b, h * G:(h + 1) * G]) - r["lse"]).max() <= 1e-4
        got = np.stack([ref.rows(cache.weights.cpu().numpy(), table[b].cpu().numpy(), int(lens[b]), 16)[h] for h in range(Hkv)])
        assert np.abs(got - np.stack(W)).max() <= 1e-4 * np.stack(W).max()


@gpu
def test_captured_step_replays_with_new_lengths():
    lens = np.array([300, 41], np.int32)
    pool = Pool(2, 2, 128, 16, [320, 320], seed=51)
    c, table, n = pool.cache(), dev(pool.table), dev(lens)
    rng = np.random.default_rng(52)
    q, kn = bf16(rng.standard_normal((2, 8, 1, 128))).cuda(), bf16(rng.standard_normal((2, 2, 1, 128))).cuda()
    ws = torch.empty(fa.fa_fwd_kv4_workspace_bytes(2, 8, 2, 1, 128, pool.cols * 16, True), dtype=torch.uint8, device="cuda")
    step = lambda cache, m: (fa.kv4_append(cache, kn, kn, m, table), fa.forward_kv4(q, cache, m, table, accumulate=True, workspace=ws))[1]  # noqa: E731
    step(pool.cache(), n.clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n.add_(1)
        o, lse = step(c, n)
    plain, m = pool.cache(), dev(lens)
    for _ in range(3):
        g.replay()
        m = m + 1
        o2, lse2 = step(plain, m)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert all(torch.equal(a, b) for a, b in zip(c, plain))
    ok()


@gpu
def test_captured_prompt_and_eviction_replay_with_new_values():
    # key weights, append, eviction and reading back in one graph, replayed with other inputs in the same places
    g = torch.Generator().manual_seed(55)
    rnd = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    B, H, Hkv, N, d, P, keep = 2, 4, 2, 300, 64, 32, 100
    q, k, v = rnd(B, H, N, d), rnd(B, Hkv, N, d), rnd(B, Hkv, N, d)
    lse, lens = torch.full((B, H, N), 6.0, device="cuda"), torch.tensor([300, 170], dtype=torch.int32, device="cuda")
    order = torch.randperm(40, generator=g).to(torch.int32).cuda()
    table, to = order[:20].view(2, 10).contiguous(), order[20:28].view(2, 4).contiguous()

    def work(cache):
        w = fa.key_weights(q, k, lse, causal=True)
        fa.kv4_append(cache, k, v, lens, table, n_new=lens, weights=w)
        kept, now = fa.kv4_evict(cache, lens, table, cache, to, keep, recent=9)
        return (kept, now, *fa.kv4_read(cache, now, to, keep))

    work(fa.kv4_cache(40, Hkv, P, d))
    torch.cuda.synchronize()
    cache, graph = fa.kv4_cache(40, Hkv, P, d), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work(cache)
    for turn in range(3):
        for t in (q, k, v):
            t.copy_(rnd(*t.shape))
        lens.copy_(torch.tensor([300 - 90 * turn, 101 + turn], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, work(fa.kv4_cache(40, Hkv, P, d))))
    ok()


@gpu
def test_given_stream_and_repeated_calls_give_the_same_bits():
    lens = np.array([3000, 77], np.int32)
    pool = Pool(2, 1, 128, 64, lens, seed=61)
    q = bf16(np.random.default_rng(62).standard_normal((2, 8, 1, 128))).cuda()
    c, table, n = pool.cache(), dev(pool.table), dev(lens)
    o, lse = fa.forward_kv4(q, c, n, table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(s):
            ws = torch.empty(fa.fa_fwd_kv4_workspace_bytes(2, 8, 1, 1, 128, table.shape[1] * 64, False), dtype=torch.uint8, device="cuda")
        o2, lse2 = fa.forward_kv4(q, c, n, table, workspace=ws, stream=s)
        s.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    ok()


@gpu
@pytest.mark.parametrize("d,G,n_q", [(128, 4, 3), (128, 16, 1), (128, 8, 4), (64, 4, 3), (64, 8, 4), (128, 4, 9)])
def test_groups_of_rows_run_apart_and_agree(d, G, n_q):
    # 9 to 36 rows a key head: two or four groups of threads share the products, each at its own pace, over many tiles;
    # calls back to back, so that the tiles come from L2 as fast as they ever do
    lens = np.array([5000, 900, 2300, 1, 3700, 130, 4096, 640], np.int32)
    pool = Pool(8, 4, d, 32, lens, seed=d + G)
    q = bf16(2 * np.random.default_rng(G).standard_normal((8, 4 * G, n_q, d))).cuda()
    c, table, n = pool.cache(), dev(pool.table), dev(lens)
    runs = [fa.forward_kv4(q, c, n, table) for _ in range(12)]
    o, lse = fa.forward_kv4(q, c, n, table, accumulate=True)
    ok()
    check_attention(pool, q, lens, fa.default_scale(d), o, lse, pool.w, f64(c.weights))
    assert all(torch.equal(o, x) and torch.equal(lse, y) for x, y in runs)


@gpu
def test_calls_on_several_streams_at_once():
    # attention with different groupings, key weights, an append and an eviction side by side: each as it is alone
    lens = np.array([2500, 60, 700], np.int32)
    pools = [Pool(3, 2, d, 32, lens, seed=91 + i) for i, d in enumerate((128, 128, 64))]
    g = torch.Generator().manual_seed(7)
    rnd = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    qs = [rnd(3, 2 * G, 1, p.d) for p, G in zip(pools, (4, 12, 24))]
    qw, kw, lse = rnd(1, 8, 1000, 128), rnd(1, 2, 1000, 128), torch.full((1, 8, 1000), 7.0, device="cuda")
    n, caches, tables = dev(lens), [p.cache() for p in pools], [dev(p.table) for p in pools]
    other = fa.kv4_cache(40, 2, 32, 128)
    to = torch.arange(30, dtype=torch.int32, device="cuda").view(3, 10)
    jobs = [lambda s, i=i: fa.forward_kv4(qs[i], caches[i], n, tables[i], stream=s) for i in range(3)]
    jobs += [lambda s: (fa.key_weights(qw, kw, lse, causal=True, stream=s),),
             lambda s: fa.kv4_evict(caches[0], n, tables[0], other, to, 300, recent=20, stream=s)]
    alone = [job(None) for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        outs = [job(s) for job, s in zip(jobs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, outs):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    ok()


@gpu
def test_sequences_may_share_pages_that_are_read():
    lens = np.array([90, 50], np.int32)
    pool = Pool(2, 1, 64, 16, lens, seed=71)
    table = pool.table.copy()
    table[1, :3] = table[0, :3]  # a common prefix of three pages
    q = bf16(np.random.default_rng(72).standard_normal((1, 2, 1, 64)))
    o, lse = fa.forward_kv4(torch.cat([q, q]).cuda(), pool.cache(), dev(np.array([48, 48], np.int32)), dev(table))
    ok()
    assert torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1])


@gpu
def test_rows_past_four_gibibytes():
    # a pool of 4.6 GB of K codes: byte offsets pass 32 bits
    d, P, Hkv = 128, 1024, 1
    n_pages = 70_000
    c = fa.kv4_cache(n_pages, Hkv, P, d)
    pages = np.array([[n_pages - 1, 0, n_pages - 2]], np.int32)
    rng = np.random.default_rng(81)
    x = bf16(rng.standard_normal((1, 1, 2100, d)))
    n = np.array([2100], np.int32)
    fa.kv4_append(c, x.cuda(), x.cuda(), dev(n), dev(pages))
    k, v = fa.kv4_read(c, dev(n), dev(pages), 2100)
    q = bf16(rng.standard_normal((1, 4, 1, d))).cuda()
    o, lse = fa.forward_kv4(q, c, dev(n), dev(pages), accumulate=True)
    to = np.array([[n_pages - 3]], np.int32)
    kept, now = fa.kv4_evict(c, dev(n), dev(pages), c, dev(to), 1000, recent=10)
    k2, _ = fa.kv4_read(c, now, dev(to), 1000)
    ok()
    kk = ref.values(*ref.quantise(f64(x[0]), 32))
    vv = ref.values(*ref.quantise(f64(x[0]), d))
    assert (f64(k[0]) == kk).all() and (f64(v[0]) == vv).all()
    r = ref.attention(f64(q[0]), kk, vv, fa.default_scale(d), 2100)
    assert np.abs(f64(o[0]) - r["o"]).max() <= 2.0 ** -8 * np.abs(r["o"]).max()
    assert torch.equal(k2[0, 0], k[0, 0][kept[0, 0].long()])
