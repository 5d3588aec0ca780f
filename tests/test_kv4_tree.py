"""Speculative decoding on the 4-bit cache: attention of a tree of drafts, the path that is kept, copies of pages.

Moved bytes are compared exactly, attention within the bounds of attention over the cache (derived at the top of
test_kv4.py: the arithmetic is the same, the masks differ).
"""
import numpy as np
import pytest
import torch

import exact_attention_32_gb300 as fa
from oracle import kv4 as ref
from oracle import packed
from test_kv4 import BAD_CACHES, Pool, _struct, bf16, dev, f64, ok

gpu = pytest.mark.gpu


def random_tree(rng, B, n_q):
    """Parents (-1: the context) and masks (int64 [B, n_q], a draft's ancestors and itself)."""
    parent = np.array([[int(rng.integers(-1, i)) for i in range(n_q)] for _ in range(B)])
    masks = np.zeros((B, n_q), np.uint64)
    for b in range(B):
        for i in range(n_q):
            masks[b, i] = np.uint64(1 << i) | (masks[b, parent[b, i]] if parent[b, i] >= 0 else np.uint64(0))
    return parent, masks.view(np.int64)


def randn_bf16(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


def check_tree(pool, q, lens, scale, masks, n_new, o, lse):
    d = q.shape[3]
    o, lse, qd = f64(o), f64(lse), f64(q)
    for b in range(len(lens)):
        n = int(lens[b])
        k, v = pool.kv(b, n)
        r = ref.tree_attention(qd[b], k, v, scale, n, [int(m) for m in masks[b]], None if n_new is None else int(n_new[b]))
        eS = (d + 8) * 2.0 ** -23 * r["reach"] + 2.0 ** -21 * r["top_q"]
        live = r["lse"] > -np.inf
        assert (lse[b][~live] == -np.inf).all() and (o[b][~live] == 0).all()
        top = np.where(live, np.abs(r["lse"]), 0)
        assert (np.abs(lse[b][live] - r["lse"][live]) <= (eS + 2.0 ** -22 * (top + 1))[live]).all()
        rel = 2 * eS + 2.0 ** -21 * (top + 2)
        tiny = n * 2.0 ** -17 * 6 * pool.largest_v_scale(b, n) / r["total"]
        tol = (rel + 2.0 ** -8)[..., None] * r["spread"] + tiny[..., None] + 2.0 ** -8 * np.abs(r["o"])
        err = np.abs(o[b] - r["o"])
        assert (err <= tol).all(), (b, (err / np.maximum(tol, 1e-300)).max())


# ------------------------------------------------------------------- the reference and refusals (CPU)

def test_reference_of_a_chain_is_the_causal_attention():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((4, 3, 8)), rng.standard_normal((2, 9, 8)), rng.standard_normal((2, 9, 8))
    a, b = ref.attention(q, k, v, 0.3, 9), ref.tree_attention(q, k, v, 0.3, 9, [1, 3, 7], None)
    assert np.array_equal(a["o"], b["o"]) and np.array_equal(a["lse"], b["lse"])
    c = ref.tree_attention(q, k, v, 0.3, 9, [1, 2, 5], 2)  # two drafts that do not see one another; no third
    e = np.exp(0.3 * k[0, [0, 1, 2, 3, 4, 5, 6, 8]] @ q[1, 1])
    assert np.isclose(c["lse"][1, 1], np.log(e.sum())) and (c["lse"][:, 2] == -np.inf).all()


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches_are_refused_before_any_device_call(kw, code):
    c, p = _struct(**kw), 1 << 20
    assert fa.fa_fwd_kv4_tree(p, c, p, p, p, None, p, p, 1, 2, 1, 1, 0.1, p, 1 << 40, 0) == code
    assert fa.fa_kv4_keep(c, p, p, 1, p, p, None, 1, 1, p, 0) == code
    assert fa.fa_kv4_copy_pages(c, p, _struct(), p, 1, 0) == code
    assert fa.fa_kv4_copy_pages(_struct(), p, c, p, 1, 0) == code


def test_bad_arguments_are_refused_before_any_device_call():
    c, p = _struct(), 1 << 20
    ws = fa.fa_fwd_kv4_tree_workspace_bytes(1, 4, 2, 3, 64, 16)

    def tree(tree=p, B=1, H=4, n_q=3, cols=1, scale=0.1, bytes=ws):
        return fa.fa_fwd_kv4_tree(p, c, p, p, tree, None, p, p, B, H, n_q, cols, scale, p, bytes, 0)
    for kw in (dict(tree=None), dict(B=0), dict(H=3), dict(H=0), dict(n_q=0), dict(n_q=65), dict(H=64, n_q=64), dict(cols=0),
               dict(cols=1 << 40), dict(scale=0.0), dict(scale=float("nan")), dict(bytes=ws - 1)):
        assert tree(**kw) == 1, kw
    for B, n, cols in ((0, 1, 1), (1, 0, 1), (1, 65, 1), (1, 1, 0), (1, 1, 1 << 40), (1 << 31, 1, 1)):
        assert fa.fa_kv4_keep(c, p, p, cols, p, p, None, B, n, p, 0) == 1
    assert fa.fa_kv4_copy_pages(c, p, _struct(page_size=32), p, 1, 0) == 1
    assert fa.fa_kv4_copy_pages(c, p, _struct(Hkv=3), p, 1, 0) == 1
    assert fa.fa_kv4_copy_pages(c, p, _struct(d=128), p, 1, 0) == 1
    for n in (0, -1, 1 << 31):
        assert fa.fa_kv4_copy_pages(c, p, c, p, n, 0) == 1
    big = _struct(Hkv=1 << 20, page_size=1024)
    assert fa.fa_kv4_copy_pages(big, p, big, p, 1, 0) == 1


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(32, 8), (8, 8), (8, 1), (6, 2), (64, 4)])
def test_a_workspace_of_the_largest_call_serves_every_smaller_one(H, Hkv, d):
    # a server allocates for its largest batch, table and number of drafts
    def need(B, n_q, tokens):
        return fa.fa_fwd_kv4_tree_workspace_bytes(B, H, Hkv, n_q, d, tokens)
    Bs, drafts = [1, 2, 3, 5, 8, 16, 40, 200], [1, 2, 3, 4, 6, 8, 9, 12, 16, 31, 32, 48, 64]
    drafts, rooms = [n for n in drafts if H // Hkv * n <= 1024], [16, 256, 512, 528, 640, 1040, 4000, 8192, 40000, 262144]
    all_of = {(B, n, t): need(B, n, t) for B in Bs for n in drafts for t in rooms}
    assert all(x > 0 for x in all_of.values())
    for (B, n, t), x in all_of.items():
        for up in ((Bs, 0, B), (drafts, 1, n), (rooms, 2, t)):
            at = up[0].index(up[2])
            if at + 1 < len(up[0]):
                larger = [B, n, t]
                larger[up[1]] = up[0][at + 1]
                assert x <= all_of[tuple(larger)], ((B, n, t), larger)


def test_python_calls_refuse_wrong_tensors():
    c = fa.kv4_cache(4, 2, 16, 64, device="cpu")
    i = torch.zeros(1, dtype=torch.int32)
    for bad in (lambda: fa.forward_kv4_tree(torch.zeros(1, 2, 1, 64).bfloat16(), c, i, i[None], i[None].long()),
                lambda: fa.kv4_keep(c, i, i[None], i[None], i), lambda: fa.kv4_copy_pages(c, i, c, i), lambda: fa.kv4_keep(1, i, i, i, i)):
        with pytest.raises(ValueError):
            bad()


# ----------------------------------------------------------------------------------- tree (GPU)

# The kernel for many rows a key head is taken where the table has room for many tokens, used or not.
rooms = pytest.mark.parametrize("room", [0, 1 << 18])


def table_of(pool, room):
    table = np.full((pool.B, max(pool.table.shape[1], room // pool.P)), -7, np.int32)
    table[:, :pool.table.shape[1]] = pool.table
    return dev(table)


@gpu
@rooms
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv,G,n_q", [(1, 1, 1), (2, 4, 2), (3, 7, 3), (1, 1, 9), (2, 3, 16), (1, 12, 5), (2, 2, 64), (1, 16, 8)])
def test_tree_over_short_and_odd_lengths(Hkv, G, n_q, d, room):
    # fewer tokens than drafts, drafts across tile and page borders, sequences that are all drafts, and counts of them
    lens = np.array([0, 1, 2, 15, 16, 17, 33, 63, 64, 65, 127, 129, 140, 255, 256, 257, 300, 321], np.int32)
    rng = np.random.default_rng(Hkv * 100 + G * 10 + n_q)
    pool = Pool(len(lens), Hkv, d, 16, lens, seed=Hkv * 100 + G * 10 + n_q)
    q = bf16(rng.standard_normal((len(lens), Hkv * G, n_q, d))).cuda()
    _, masks = random_tree(rng, len(lens), n_q)
    c = pool.cache()
    counts = rng.integers(-1, n_q + 2, len(lens)).astype(np.int32)
    for n_new in (None, counts):
        o, lse = fa.forward_kv4_tree(q, c, dev(lens), table_of(pool, room), dev(masks), n_new=None if n_new is None else dev(n_new))
        ok()
        check_tree(pool, q, lens, fa.default_scale(d), masks, n_new, o, lse)


@gpu
@rooms
@pytest.mark.parametrize("d,P,Hkv,G,n_q", [(128, 64, 2, 4, 12), (64, 32, 1, 8, 4), (128, 1024, 1, 1, 3), (128, 16, 1, 2, 64), (64, 128, 2, 5, 13)])
def test_tree_over_long_ragged_lengths(d, P, Hkv, G, n_q, room):
    lens = np.array([9000, 4097, 70, 700, 8192], np.int32)
    rng = np.random.default_rng(d + P)
    pool = Pool(5, Hkv, d, P, lens, seed=d + P)
    q = bf16(3 * rng.standard_normal((5, Hkv * G, n_q, d))).cuda()
    _, masks = random_tree(rng, 5, n_q)
    n_new = np.array([n_q, 1, n_q, 0, max(1, n_q - 2)], np.int32)
    o, lse = fa.forward_kv4_tree(q, pool.cache(), dev(lens), table_of(pool, room), dev(masks), n_new=dev(n_new), scale=0.11)
    ok()
    check_tree(pool, q, lens, float(np.float32(0.11)), masks, n_new, o, lse)


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n_q", [(5, 8), (4, 16), (3, 32)])
def test_many_short_caches(G, n_q, d):
    # tables of 512 tokens: items go to CTAs whole, several to each, of chunks of 48, 32 and 48 rows in the kernel for many rows
    B, Hkv, P = 80, 4, 16
    rng = np.random.default_rng(d + n_q)
    lens = rng.integers(0, 513, B).astype(np.int32)
    lens[:6] = [512, 0, 1, 511, 128, 129]
    pool = Pool(B, Hkv, d, P, lens, seed=d + n_q)
    q = bf16(rng.standard_normal((B, Hkv * G, n_q, d))).cuda()
    _, masks = random_tree(rng, B, n_q)
    n_new = rng.integers(0, n_q + 1, B).astype(np.int32)
    c, table = pool.cache(), dev(pool.table[:, :512 // P])
    for new in (None, n_new):
        o, lse = fa.forward_kv4_tree(q, c, dev(lens), table, dev(masks), n_new=None if new is None else dev(new))
        ok()
        check_tree(pool, q, lens, fa.default_scale(d), masks, new, o, lse)


@gpu
@rooms
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,n_q", [(2, 5), (5, 8), (4, 16)])
def test_rows_of_very_different_size(d, G, n_q, room):
    # the bounds are each row's own: what is rounded under the largest value of other rows would pass them
    lens = np.array([200, 700], np.int32)
    rng = np.random.default_rng(d + n_q)
    pool = Pool(2, 2, d, 32, lens, seed=d + n_q)
    q = bf16(rng.standard_normal((2, 2 * G, n_q, d)) * 2.0 ** rng.integers(-30, 4, (2, 2 * G, n_q, 1))).cuda()
    _, masks = random_tree(rng, 2, n_q)
    for gain in (1.0, 2.0 ** 24):
        o, lse = fa.forward_kv4_tree(q * gain, pool.cache(), dev(lens), table_of(pool, room), dev(masks), scale=float(0.125 / gain))
        ok()
        check_tree(pool, q * gain, lens, 0.125 / gain, masks, None, o, lse)


@gpu
@rooms
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [-1e33, 1e33, -1e-30])
def test_scores_of_any_size(size, d, room):
    # 24 rows over three tokens of a context and a draft, whose keys are 1, 2, 3 and 4 in every channel: all scores
    # far below or above zero, or next to it; the largest takes all, or all are alike
    B, G, n_q, P = 3, 8, 3, 16
    cache = fa.kv4_cache(4, 1, P, d)
    k = (torch.arange(1, 5).view(4, 1) * torch.ones(d)).bfloat16().cuda().expand(B, 1, 4, d).contiguous()
    v = randn_bf16((B, 1, 4, d), 3).cuda()
    table = np.full((B, max(1, room // P)), -7, np.int32)
    table[:, 0] = [2, 0, 3]
    table, lens = dev(table), dev(np.full(B, 4, np.int32))
    fa.kv4_append(cache, k, v, lens, table)
    ks, vs = (f64(t) for t in fa.kv4_read(cache, lens, table, 4))
    q = torch.full((B, G, n_q, d), size).bfloat16().cuda()
    masks = np.tile(np.array([1, 1, 1], np.int64), (B, 1))
    o, lse = fa.forward_kv4_tree(q, cache, lens, table, dev(masks), n_new=dev(np.ones(B, np.int32)))
    ok()
    s = float(q[0, 0, 0, 0]) * fa.default_scale(d) * ks[:, 0].sum(-1)  # [B, 4]
    e = np.exp(s - s.max(-1, keepdims=True))
    want_lse, want = s.max(-1) + np.log(e.sum(-1)), np.einsum("bn,bnd->bd", e / e.sum(-1, keepdims=True), vs[:, 0])
    for b in range(B):
        # |lse| to (d + 8) roundings of the sum and the two of its last product; O to bf16's and P's (a half) roundings
        assert (np.abs(f64(lse)[b, :, 0] - want_lse[b]) <= (d + 16) * 2.0 ** -23 * np.abs(want_lse[b]) + 1e-6).all()
        assert (np.abs(f64(o)[b, :, 0] - want[b]) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(vs[b, 0]).max(0)).all()
        assert (f64(lse)[b, :, 1:] == -np.inf).all() and (f64(o)[b, :, 1:] == 0).all()


V_SCALES = [2.0 ** -17, 2.0 ** -15, 2.0 ** -10, 2.0 ** -9, 0.3125, 0.4375, 0.5, 1.0, 1.75, 12.0, 1024.0, 10240.0]
# log2 of the largest score's magnitude (log2 units): a step of fp32 is as large as, or larger than, what separates a
# row's reference from its largest term (3 to 60) from 2^25 on
SIZES = [-31.2, -29.5, -28.4, -27.6, -26.5, 25.3, 26.5, 27.2, 27.8, 28.3, 28.8, 29.5, 30.5, 60.0]


def check_scores_under_v_scales(call, size, d, H, n_q, room, N):
    """Sequences of N tokens, keys 1, 1, 4 and 4 in every channel of a quarter of them each, V scales of one
    size or of two in turn; all queries alike, so that log2 scores reach +-2^size: half of the tokens tie and the others
    weigh nothing.  Their V are a code of at most 6 under the scale, 6 itself once at least."""
    rng = np.random.default_rng(N)
    pairs = [(s, s) for s in V_SCALES] + list(zip(V_SCALES, V_SCALES[::-1]))
    B, P = len(pairs), 16
    cols = -(-N // P)
    cache = fa.kv4_cache(B * cols, 1, P, d)
    key = np.repeat(np.array([1.0, 1.0, 4.0, 4.0]), N // 4)
    k = bf16(np.tile(key[None, None, :, None], (B, 1, 1, d))).cuda()
    v = ref.E2M1[rng.integers(0, 8, (B, 1, N, d))] * rng.choice([-1.0, 1.0], (B, 1, N, d))
    v[..., 0] = 6.0
    v *= np.array([[p[j % 2] for j in range(N)] for p in pairs])[:, None, :, None]
    table = np.full((B, max(cols, room // P)), -7, np.int32)
    table[:, :cols] = np.arange(B * cols).reshape(B, cols)
    table, lens = dev(table), dev(np.full(B, N, np.int32))
    fa.kv4_append(cache, k, bf16(v).cuda(), lens, table)
    ks, vs = (f64(t) for t in fa.kv4_read(cache, lens, table, N))
    assert (vs == v).all()
    scale = fa.default_scale(d)
    q = bf16(np.full((B, H, n_q, d), np.sign(size) * 2.0 ** abs(size) * np.log(2) / ((4 if size > 0 else 1) * d * scale))).cuda()
    o, lse = call(q, cache, lens, table)
    ok()
    s = float(q[0, 0, 0, 0]) * scale * ks[:, 0].sum(-1)  # [B, N]
    e = np.exp(s - s.max(-1, keepdims=True))
    want_lse, want = s.max(-1) + np.log(e.sum(-1)), np.einsum("bn,bnd->bd", e / e.sum(-1, keepdims=True), vs[:, 0])
    o, lse = f64(o), f64(lse)
    # |lse| to (d + 8) roundings of the sum and the two of its last product.  O to bf16's rounding and P's, of itself (a half's,
    # 2^-11) and of the smallest step.  P times V's scale is a half that is off by at most 2^-25 near its smallest step.  With many rows:
    # the row's reference r is at least x - L (x a tie's score, L = 15 - log2 of its V scale), at most one step u of fp32 at x
    # and 8 (headroom, rounded up to a whole number or a step) above that for the tie it is set by.  u <= 8: that tie's term is
    # 2^(15 - u - 8) or more; u = 16, where the headroom is lost in x's rounding, 2^(15 - 16): at least 2^-1 both, and 2^-25 is
    # 2^-24 of it.  u >= 32: r is at most x, so p is a power of two from 1 on, and p times a scale (a multiple of 2^-17) is
    # exact.  With few rows the largest term is kept between 2^11 and 2^15 and the parts are off by 2^-34 of it.  So a term is off by at
    # most 2^-24 of the largest, p max(V scale), which after the division by sum p >= p is 2^-24 max(V scale), times a code of
    # at most 6.
    assert np.isfinite(o).all() and np.isfinite(lse).all()
    for b in range(B):
        assert (np.abs(lse[b] - want_lse[b]) <= (d + 16) * 2.0 ** -23 * np.abs(want_lse[b]) + 1e-6).all(), pairs[b]
        assert (np.abs(o[b] - want[b]) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(vs[b, 0]).max(0) + 6 * 2.0 ** -24 * max(pairs[b])).all(), pairs[b]


def tree_of_alike(q, cache, lens, table):
    """The newest n_q tokens as drafts that every row admits."""
    masks = torch.full(q.shape[::2], (1 << q.shape[2]) - 1, dtype=torch.int64, device="cuda")
    return fa.forward_kv4_tree(q, cache, lens, table, masks)


@gpu
@pytest.mark.parametrize("N", [4, 600])
@pytest.mark.parametrize("d,H,n_q", [(128, 8, 3), (128, 16, 3), (64, 16, 3)])
@pytest.mark.parametrize("size", SIZES)
def test_large_scores_under_any_v_scale_with_many_rows(size, d, H, n_q, N):
    check_scores_under_v_scales(tree_of_alike, size, d, H, n_q, 1 << 18, N)


@gpu
@pytest.mark.parametrize("N", [4, 600])
@pytest.mark.parametrize("d,H,n_q,room", [(128, 1, 1, 0), (64, 4, 2, 0), (128, 8, 3, 0), (64, 8, 3, 1 << 18)])
@pytest.mark.parametrize("size", SIZES)
def test_large_scores_under_any_v_scale_with_few_rows(size, d, H, n_q, room, N):
    check_scores_under_v_scales(tree_of_alike, size, d, H, n_q, room, N)
    if n_q == 1:
        check_scores_under_v_scales(fa.forward_kv4, size, d, H, n_q, room, N)


@gpu
@rooms
@pytest.mark.parametrize("d,G,n_q", [(64, 4, 3), (128, 8, 1), (64, 2, 4), (128, 2, 16), (64, 3, 7)])
def test_a_chain_gives_the_causal_call(d, G, n_q, room):
    # bit for bit up to 8 rows a key head; above that in other chunks or another kernel's sums, within the same bounds
    lens = np.array([n_q, 500, 2000, 129, n_q + 1], np.int32)
    rng = np.random.default_rng(n_q)
    pool = Pool(5, 2, d, 32, lens, seed=n_q)
    q = bf16(rng.standard_normal((5, 2 * G, n_q, d))).cuda()
    chain = dev(np.tile(np.array([(2 << t) - 1 for t in range(n_q)], np.int64), (5, 1)))
    c = pool.cache()
    a = fa.forward_kv4(q, c, dev(lens), table_of(pool, room))
    b = fa.forward_kv4_tree(q, c, dev(lens), table_of(pool, room), chain)
    ok()
    if G * n_q <= 8:
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for o, lse in (a, b):
        check_tree(pool, q, lens, fa.default_scale(d), chain.cpu().numpy(), None, o, lse)


@gpu
@rooms
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [2, 8])
def test_masks_are_taken_as_they_are(d, G, room):
    # none, all, only others, bits behind the drafts; a stored NaN among the drafts reaches the rows that admit it
    n_q, lens = 6, np.array([6, 40, 300], np.int32)
    pool = Pool(3, 1, d, 16, lens, seed=3)
    for b in range(3):
        j = lens[b] - 2  # draft 4
        pool.ks[pool.table[b, j // 16], :, j % 16] = 255
    masks = np.tile(np.array([0, 0x2F, 0x2, -1 ^ 0x10, 0x3F, (1 << 63) - 1 - 0x10], np.int64), (3, 1))
    q = bf16(np.random.default_rng(4).standard_normal((3, G, n_q, d))).cuda()
    o, lse = fa.forward_kv4_tree(q, pool.cache(), dev(lens), table_of(pool, room), dev(masks))
    ok()
    assert torch.isnan(lse[:, :, 4]).all() and (lse[0, :, 0] == -np.inf).all() and (o[0, :, 0] == 0).all()
    rest = [0, 1, 2, 3, 5]
    assert not torch.isnan(o[:, :, rest]).any() and not torch.isnan(lse[:, :, rest]).any()
    for b in range(3):  # (draft 4 is finite again for the reference, which the other rows do not see)
        j = lens[b] - 2
        pool.ks[pool.table[b, j // 16], :, j % 16] = 0
    check = [0, 1, 2, 3, 5]
    for b in range(3):
        n = int(lens[b])
        k, v = pool.kv(b, n)
        r = ref.tree_attention(f64(q)[b], k, v, fa.default_scale(d), n, [int(m) for m in masks[b]], None)
        live = r["lse"][:, check] > -np.inf
        assert np.abs(f64(lse)[b][:, check][live] - r["lse"][:, check][live]).max() <= 1e-4
        assert np.abs(f64(o)[b][:, check] - r["o"][:, check]).max() <= 2.0 ** -6 * np.abs(v).max()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_tree_in_the_workspace_of_a_larger_batch(d):
    # and no byte behind it is touched, of a small batch's chunks and of a large one's
    H, Hkv, n_q, room, P = 32, 8, 6, 8192, 64
    need = fa.fa_fwd_kv4_tree_workspace_bytes(16, H, Hkv, n_q, d, room)
    ws = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    for B in (3, 16):
        lens = np.array([200, 9, 700, 0, 64] * 4, np.int32)[:B]
        rng = np.random.default_rng(B + d)
        pool = Pool(B, Hkv, d, P, lens, seed=B + d)
        q = bf16(rng.standard_normal((B, H, n_q, d))).cuda()
        _, masks = random_tree(rng, B, n_q)
        o, lse = fa.forward_kv4_tree(q, pool.cache(), dev(lens), table_of(pool, room), dev(masks), workspace=ws[:need])
        ok()
        check_tree(pool, q, lens, fa.default_scale(d), masks, None, o, lse)
    assert (ws[need:] == 171).all()


@gpu
def test_tree_refuses_wrong_gpu_tensors():
    pool = Pool(2, 2, 64, 16, [40, 20], seed=5)
    c, lens, table = pool.cache(), dev(np.array([40, 20], np.int32)), dev(pool.table)
    q, masks = torch.zeros(2, 4, 3, 64, device="cuda").bfloat16(), torch.ones(2, 3, dtype=torch.int64, device="cuda")
    for bad in (dict(tree=masks.int()), dict(tree=masks[:, :2]), dict(tree=masks[:1]), dict(tree=masks.cpu()), dict(tree=masks.T),
                dict(n_new=lens.long()), dict(n_new=lens[:1]), dict(q=q[:, :3])):
        a = {**dict(q=q, cache=c, lens=lens, page_table=table, tree=masks), **bad}
        with pytest.raises(ValueError):
            fa.forward_kv4_tree(**a)
    with pytest.raises(fa.FAError):
        fa.forward_kv4_tree(q, c, lens, table, masks, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    ok()


@gpu
@rooms
@pytest.mark.parametrize("G", [2, 8])
def test_tree_leaves_bad_pages_out_and_reports_them(G, room):
    lens = np.array([100, 60], np.int32)
    pool = Pool(2, 1, 64, 16, lens, seed=6)
    q = bf16(np.random.default_rng(7).standard_normal((2, G, 4, 64))).cuda()
    _, masks = random_tree(np.random.default_rng(8), 2, 4)
    table = table_of(pool, room)
    table[0, 6] = pool.n_pages  # holds tokens 96 .. 99: all four drafts
    o, lse = fa.forward_kv4_tree(q, pool.cache(), dev(lens), table, dev(masks))
    torch.cuda.synchronize()
    assert fa.fa_get_device_status(0) == 8
    k, v = pool.kv(0, 96)
    r = ref.tree_attention(f64(q)[0], np.concatenate([k, k[:, :4]], 1),
                           np.concatenate([v, v[:, :4]], 1), fa.default_scale(64), 100, [0] * 4, None)
    assert np.abs(f64(lse)[0] - r["lse"]).max() <= 1e-4
    ok()


# ----------------------------------------------------------------------------------- keep (GPU)

def pool_arrays(c):
    return [t.cpu().numpy() for t in c]


def kept(pool, lens, path, n_path, n_new, S):
    """The pool's arrays after keeping, and the new lengths."""
    arrays = [x.copy() for x in (pool.k, pool.v, pool.ks, pool.vs, pool.w)]
    now = []
    for b in range(pool.B):
        n = int(lens[b])
        drafts = min(S, n) if n_new is None else min(max(int(n_new[b]), 0), min(S, n))
        m = min(max(int(n_path[b]), 0), drafts)
        p, good = [int(x) for x in path[b]], []
        for x in p[:m]:
            if x >= drafts or x <= (good[-1] if good else -1):
                break
            good.append(x)
        at = lambda j: (pool.table[b, (n - drafts + j) // pool.P], slice(None), (n - drafts + j) % pool.P)  # noqa: E731
        for x in arrays:
            rows = [x[at(j)].copy() for j in good]
            for i, row in enumerate(rows):
                x[at(i)] = row
        now.append(n - drafts + len(good))
    return arrays, now


@gpu
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("Hkv,d,P,S", [(1, 64, 16, 1), (3, 128, 16, 64), (2, 64, 32, 7), (2, 128, 64, 33), (1, 64, 1024, 64), (5, 128, 16, 12)])
def test_keep_moves_the_path_and_nothing_else(Hkv, d, P, S, weights):
    lens = np.array([0, 1, S, S + 1, 100, 300, 129, 200, S // 2], np.int32)
    rng = np.random.default_rng(S)
    pool = Pool(len(lens), Hkv, d, P, np.maximum(lens, 1), seed=S)
    pool.ks[:], pool.vs[:] = rng.integers(0, 256, pool.ks.shape), rng.integers(0, 256, pool.vs.shape)  # every byte moves as it is
    path = np.zeros((len(lens), S), np.int32)
    for b in range(len(lens)):
        path[b] = np.sort(rng.permutation(S))
        some = np.sort(rng.permutation(S)[:max(1, S // 2)])
        path[b, :len(some)] = some
    n_path = rng.integers(-1, S + 2, len(lens)).astype(np.int32)
    n_path[4:] = np.minimum(n_path[4:], max(1, S // 2))
    for n_new in (None, rng.integers(-1, S + 2, len(lens)).astype(np.int32)):
        want, now = kept(pool, lens, path, n_path, n_new, S)
        c = pool.cache()
        if not weights:
            c = c._replace(weights=None)
        got = fa.kv4_keep(c, dev(lens), dev(pool.table), dev(path), dev(n_path), n_new=None if n_new is None else dev(n_new))
        torch.cuda.synchronize()
        fa.fa_get_device_status(0)  # (random paths that break are reported)
        assert got.tolist() == now
        for x, y in zip(c[:4], want):
            assert np.array_equal(x.cpu().numpy(), y)
        if weights:
            assert np.array_equal(c.weights.cpu().numpy(), want[4])


@gpu
def test_keep_reports_paths_that_do_not_ascend_and_only_those():
    lens = np.array([50, 60, 70, 80], np.int32)
    pool = Pool(4, 2, 64, 16, lens, seed=9)
    good = np.array([[0, 2, 3, 0], [1, 3, 0, 0], [0, 1, 2, 3], [9, 9, 9, 9]], np.int32)
    for path, n_path, status, now in ((good, [3, 2, 4, 0], 0, [49, 58, 70, 76]), (good, [4, 2, 4, 0], 8, [49, 58, 70, 76]),
                                      (good, [3, 3, 4, 1], 8, [49, 58, 70, 76]), (good - 1, [3, 2, 4, 0], 8, [46, 58, 66, 76]),
                                      (np.array([[2 ** 31 - 1] * 4, [-2 ** 31] * 4, [3, 3, 3, 3], [0, 4, 5, 6]], np.int32), [4] * 4, 8,
                                       [46, 56, 67, 77])):
        n_path = np.array(n_path, np.int32)
        want, expect = kept(pool, lens, np.where(path < 0, 99, path), n_path, None, 4)
        c = pool.cache()
        got = fa.kv4_keep(c, dev(lens), dev(pool.table), dev(path), dev(n_path))
        torch.cuda.synchronize()
        assert fa.fa_get_device_status(0) == status and got.tolist() == expect == now
        assert all(np.array_equal(x, y) for x, y in zip(pool_arrays(c), want))


@gpu
def test_keep_with_bad_pages():
    lens = np.array([36, 36], np.int32)
    pool = Pool(2, 1, 64, 16, lens, seed=10)
    table = pool.table.copy()
    table[0, 1], table[1, 2] = -1, pool.n_pages  # tokens 16 .. 31 of the first, 32 .. 35 of the second
    path = np.array([[5, 6, 7, 0, 0, 0, 0, 0]] * 2, np.int32)
    c = pool.cache()
    before = pool_arrays(c)
    got = fa.kv4_keep(c, dev(lens), dev(table), dev(path), dev(np.array([3, 3], np.int32)))
    torch.cuda.synchronize()
    assert fa.fa_get_device_status(0) == 8 and got.tolist() == [31, 31]
    after = pool_arrays(c)
    # the first's path (33, 34, 35) would go to 28 .. 30, in no page: nothing is written.  The second's comes from no page: zeros
    for x, y in zip(before, after):
        want = x.copy()
        want[table[1, 1], :, 12:15] = 0
        assert np.array_equal(y, want)
    ok()


@gpu
def test_keep_refuses_wrong_gpu_tensors():
    pool = Pool(2, 2, 64, 16, [40, 20], seed=5)
    c, lens, table = pool.cache(), dev(np.array([40, 20], np.int32)), dev(pool.table)
    path = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    for bad in (dict(path=path.long()), dict(path=path[:1]), dict(path=path[:, :0]), dict(path=torch.zeros(2, 65).int().cuda()),
                dict(n_path=lens[:1]), dict(n_path=lens.cpu()), dict(n_new=lens.long()), dict(lens=lens[:1])):
        with pytest.raises(ValueError):
            fa.kv4_keep(**{**dict(cache=c, lens=lens, page_table=table, path=path, n_path=lens), **bad})
    assert fa.fa_kv4_keep(fa.KV4CacheStruct(*[t.data_ptr() for t in c], pool.n_pages, 2, 16, 64), lens.data_ptr(), table.data_ptr(),
                          pool.cols, path.data_ptr(), lens.data_ptr(), None, 2, 4, lens.data_ptr(), 0) == 1  # new_lens over lens
    ok()


# ----------------------------------------------------------------------------------- copy (GPU)

@gpu
@pytest.mark.parametrize("Hkv,d,P,n", [(1, 64, 16, 1), (3, 128, 16, 40), (8, 128, 64, 30), (5, 64, 1024, 3), (2, 64, 32, 500)])
@pytest.mark.parametrize("same_pool", [True, False])
def test_copies_are_the_pages_and_nothing_else(same_pool, Hkv, d, P, n):
    g = torch.Generator().manual_seed(n)
    N = 2 * n + 3

    def cache(pages):
        c = fa.kv4_cache(pages, Hkv, P, d, device="cpu")
        return fa.KV4Cache(*[torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8) if t.dtype == torch.uint8
                             else torch.randn(t.shape, generator=g) for t in c])
    a, b = cache(N), cache(N + 1)
    order = torch.randperm(N, generator=g).int()
    src, dst = order[:n].clone(), order[n:2 * n].clone()
    src[n // 2] = src[0]  # one page to two others
    if n > 3:
        src[1], dst[2] = -1, -5
    to = a if same_pool else b
    want = [t.clone() for t in to]
    for s, t in zip(src.tolist(), dst.tolist()):
        if s >= 0 and t >= 0:
            for x, y in zip(want, a):
                x[t] = y[s]
    ca = fa.KV4Cache(*[t.cuda() for t in a])
    ct = ca if same_pool else fa.KV4Cache(*[t.cuda() for t in b])
    fa.kv4_copy_pages(ca, src.cuda(), ct, dst.cuda())
    ok()
    for x, y in zip(ct, want):
        assert np.array_equal(x.cpu().numpy().view(np.uint8), y.numpy().view(np.uint8))
    if not same_pool:
        assert all(torch.equal(x.cpu(), y) for x, y in zip(ca, a))


@gpu
def test_copies_between_caches_with_and_without_weights():
    a, b = fa.kv4_cache(4, 2, 16, 64), fa.kv4_cache(4, 2, 16, 64)
    for t in (*a, *b):
        t.fill_(3)
    i = torch.tensor([1], dtype=torch.int32, device="cuda")
    j = torch.tensor([2], dtype=torch.int32, device="cuda")
    fa.kv4_copy_pages(a._replace(weights=None), i, b, j)
    fa.kv4_copy_pages(b, i, a._replace(weights=None), j)
    ok()
    assert (b.weights[2] == 0).all() and (b.weights[[0, 1, 3]] == 3).all() and (a.weights == 3).all()


@gpu
def test_copies_of_pages_past_the_pool_are_left_out_and_reported():
    a = fa.kv4_cache(4, 1, 16, 64)
    a.k.copy_(torch.arange(4, device="cuda").view(4, 1, 1, 1).expand_as(a.k))
    for src, dst in (([4, 0], [2, 3]), ([1, 0], [4, 3]), ([2 ** 31 - 1, 0], [1, 3])):
        a.k[3] = 9
        fa.kv4_copy_pages(a, torch.tensor(src).int().cuda(), a, torch.tensor(dst).int().cuda())
        torch.cuda.synchronize()
        assert fa.fa_get_device_status(0) == 8 and a.k[:, 0, 0, 0].tolist() == [0, 1, 2, 0]
    fa.kv4_copy_pages(a, torch.tensor([-1]).int().cuda(), a, torch.tensor([7]).int().cuda())
    fa.kv4_copy_pages(a, torch.zeros(0).int().cuda(), a, torch.zeros(0).int().cuda())
    ok()
    i = torch.zeros(2).int().cuda()
    for bad in (lambda: fa.kv4_copy_pages(a, i, a, i[:1]), lambda: fa.kv4_copy_pages(a, i.long(), a, i), lambda: fa.kv4_copy_pages(a, i.cpu(), a, i),
                lambda: fa.kv4_copy_pages(a, i, fa.kv4_cache(4, 2, 16, 64), i)):
        with pytest.raises(ValueError):
            bad()
    # arrays that meet out of step: a pool one page into the other's memory
    k = torch.zeros(5, 1, 16, 32, dtype=torch.uint8, device="cuda")
    with pytest.raises(fa.FAError):
        fa.kv4_copy_pages(a._replace(k=k[:4]), i, a._replace(k=k[1:]), i)


@gpu
def test_pages_past_four_gibibytes():
    c = fa.kv4_cache(70000, 8, 128, 128, weights=False)  # 64 KB of K a page: 4.6 GB
    last = torch.tensor([69999], dtype=torch.int32, device="cuda")
    c.k[69999], c.v[69999], c.k_scale[69999], c.v_scale[69999] = 1, 2, 3, 4
    for to in (69998, 3):
        fa.kv4_copy_pages(c, last, c, torch.tensor([to], dtype=torch.int32, device="cuda"))
        ok()
        for t, x in zip(c[:4], (1, 2, 3, 4)):
            assert (t[to] == x).all() and (t[to - 1] == 0).all()


@gpu
@rooms
def test_trees_and_kept_paths_past_four_gibibytes(room):
    # the pages of two sequences at the end of a pool of 4.6 GB of K
    lens, Hkv, G, n_q, d, P = np.array([400, 130], np.int32), 8, 6, 8, 128, 128
    pool = Pool(2, Hkv, d, P, lens, seed=77)
    first = 70000 - pool.n_pages
    c = fa.kv4_cache(70000, Hkv, P, d)
    for big, small in zip(c, (pool.k, pool.v, pool.ks, pool.vs, pool.w)):
        big[first:] = dev(small)
    rng = np.random.default_rng(78)
    q = bf16(rng.standard_normal((2, Hkv * G, n_q, d))).cuda()
    _, masks = random_tree(rng, 2, n_q)
    table = table_of(pool, room)
    table += torch.where(table >= 0, first, 0).int()
    o, lse = fa.forward_kv4_tree(q, c, dev(lens), table, dev(masks))
    ok()
    check_tree(pool, q, lens, fa.default_scale(d), masks, None, o, lse)
    path, n_path = np.tile(np.array([1, 2, 5, 7, 0, 0, 0, 0], np.int32), (2, 1)), np.array([4, 3], np.int32)
    got = fa.kv4_keep(c, dev(lens), table, dev(path), dev(n_path))
    ok()
    want, now = kept(pool, lens, path, n_path, None, n_q)
    assert got.tolist() == now
    for big, small in zip(c, want):
        assert np.array_equal(big[first:].cpu().numpy(), small) and not big[first - 4:first].any()


# ------------------------------------------------------------------------- as they are used together (GPU)

def speculate(prompts, H, Hkv, d, P, forks, drafts, tree, path, seed):
    """Packed prompts into the cache, `forks` continuations of each, a tree of drafts verified, the path kept, one token
    behind it.  Returns every tensor that the reference needs."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g).bfloat16().cuda()  # noqa: E731
    B, S = len(prompts), len(prompts) * forks
    cu = np.concatenate([[0], np.cumsum(prompts)])
    T, n = int(cu[-1]), max(prompts)
    qkv = rnd(T, H + 2 * Hkv, d)
    o, lse = fa.forward_packed(qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], dev(cu.astype(np.int32)), causal=True)
    cols = -(-(n + drafts + 1) // P)
    cache = fa.kv4_cache(B * cols + S * cols, Hkv, P, d)
    table = torch.arange(B * cols, dtype=torch.int32, device="cuda").view(B, cols)
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    at = torch.tensor(cu[:-1], device="cuda")[:, None] + torch.arange(n, device="cuda")
    rows = qkv[at.clamp(max=T - 1)].transpose(1, 2)  # [B, heads, n, d]; what lies behind a prompt is not appended
    fa.kv4_append(cache, rows[:, H:H + Hkv].contiguous(), rows[:, H + Hkv:].contiguous(), lens, table, n_new=lens)
    # a fork shares its parent's full pages, copies the page that it goes on in, and has the others for itself
    new = torch.arange(B * cols, (B + S) * cols, dtype=torch.int32, device="cuda").view(S, cols)
    flens, ftable = lens.repeat_interleave(forks), table.repeat_interleave(forks, 0)
    page = (flens // P)[:, None]
    ftable = torch.where(torch.arange(cols, device="cuda")[None] < page, ftable, new).contiguous()
    fa.kv4_copy_pages(cache, table.repeat_interleave(forks, 0).gather(1, page.long())[:, 0].contiguous(), cache,
                      new.gather(1, page.long())[:, 0].contiguous())
    dk, dv, dq = rnd(S, Hkv, drafts, d), rnd(S, Hkv, drafts, d), rnd(S, H, drafts, d)
    flens = flens + drafts
    fa.kv4_append(cache, dk, dv, flens, ftable)
    to, tl = fa.forward_kv4_tree(dq, cache, flens, ftable, tree)
    flens = fa.kv4_keep(cache, flens, ftable, path, (path >= 0).sum(1).int())
    k1, v1, q1 = rnd(S, Hkv, 1, d), rnd(S, Hkv, 1, d), rnd(S, H, 1, d)
    flens = flens + 1
    fa.kv4_append(cache, k1, v1, flens, ftable)
    no, nl = fa.forward_kv4(q1, cache, flens, ftable)
    return dict(qkv=qkv, cu=cu, o=o, lse=lse, dk=dk, dv=dv, dq=dq, to=to, tl=tl, k1=k1, v1=v1, q1=q1, no=no, nl=nl, lens=flens, cache=cache,
                table=table)


@gpu
@pytest.mark.parametrize("H,Hkv,d,P", [(8, 2, 128, 16), (6, 3, 64, 32)])
def test_prompt_fork_draft_verify_keep_and_go_on(H, Hkv, d, P):
    prompts, forks, drafts = [70, 1, 33, 64], 3, 10
    S = len(prompts) * forks
    rng = np.random.default_rng(d)
    parent, masks = random_tree(rng, S, drafts)
    path = np.full((S, drafts), -1, np.int32)
    for s in range(S):
        node, way = int(rng.integers(0, drafts)), []
        while node >= 0:
            way.append(node)
            node = int(parent[s, node])
        path[s, :len(way)] = way[::-1]
    r = speculate(prompts, H, Hkv, d, P, forks, drafts, dev(masks), dev(path), seed=d)
    ok()
    qkv, scale, G = f64(r["qkv"]), fa.default_scale(d), H // Hkv
    p = packed.forward(qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], r["cu"], scale, True)
    assert np.abs(f64(r["o"]) - p["o"]).max() <= 2.0 ** -6 * np.abs(qkv[:, H + Hkv:]).max() and np.abs(f64(r["lse"]) - p["lse"]).max() <= 1e-4
    stored = lambda x, block: ref.values(*ref.quantise(x, block))  # noqa: E731
    for s in range(S):
        a, e = r["cu"][s // forks], r["cu"][s // forks + 1]
        k = stored(qkv[a:e, H:H + Hkv].transpose(1, 0, 2), 32)
        v = stored(qkv[a:e, H + Hkv:].transpose(1, 0, 2), d)
        dk, dv = stored(f64(r["dk"][s]), 32), stored(f64(r["dv"][s]), d)
        t = ref.tree_attention(f64(r["dq"][s]), np.concatenate([k, dk], 1), np.concatenate([v, dv], 1), scale, e - a + drafts,
                               [int(m) for m in masks[s]], None)
        assert np.abs(f64(r["tl"][s]) - t["lse"]).max() <= 1e-4
        assert np.abs(f64(r["to"][s]) - t["o"]).max() <= 2.0 ** -6 * np.abs(t["spread"]).max()
        way = path[s][path[s] >= 0]
        k = np.concatenate([k, dk[:, way], stored(f64(r["k1"][s]), 32)], 1)
        v = np.concatenate([v, dv[:, way], stored(f64(r["v1"][s]), d)], 1)
        assert int(r["lens"][s]) == k.shape[1]
        t = ref.attention(f64(r["q1"][s]), k, v, scale, k.shape[1])
        assert np.abs(f64(r["nl"][s]) - t["lse"]).max() <= 1e-4
        assert np.abs(f64(r["no"][s]) - t["o"]).max() <= 2.0 ** -6 * np.abs(t["spread"]).max()
    # the prompts' own pages are as the append left them
    k, v = fa.kv4_read(r["cache"], dev(np.array(prompts, np.int32)), r["table"], 70)
    for b, n in enumerate(prompts):
        a = r["cu"][b]
        assert np.array_equal(f64(k)[b, :, :n], stored(qkv[a:a + n, H:H + Hkv].transpose(1, 0, 2), 32))


@gpu
def test_captured_verification_replays_with_new_drafts():
    rng = np.random.default_rng(12)
    S, H, Hkv, n_q, d, P = 3, 8, 2, 6, 64, 16
    pool = Pool(S, Hkv, d, P, [200, 40, 90], seed=13)
    c, table = pool.cache(), dev(pool.table)
    lens, n_path = dev(np.array([190, 30, 77], np.int32)), dev(np.array([1, 1, 1], np.int32))
    q, k = (bf16(rng.standard_normal((S, h, n_q, d))).cuda() for h in (H, Hkv))
    tree, path = dev(random_tree(rng, S, n_q)[1]), dev(np.tile(np.arange(n_q, dtype=np.int32), (S, 1)))

    def step(cache):
        fa.kv4_append(cache, k, k, lens, table)
        o, lse = fa.forward_kv4_tree(q, cache, lens, table, tree)
        return o, lse, fa.kv4_keep(cache, lens, table, path, n_path)
    step(pool.cache())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(c)
    plain = pool.cache()
    for turn in range(3):
        q.copy_(bf16(rng.standard_normal(q.shape)))
        tree.copy_(dev(random_tree(rng, S, n_q)[1]))
        path.copy_(dev(np.sort(np.array([rng.permutation(n_q) for _ in range(S)]), 1).astype(np.int32)))
        path[:, 0] = turn
        path[:, 1:] += turn * (path[:, 1:] > 0)
        graph.replay()
        got = step(plain)
        torch.cuda.synchronize()
        fa.fa_get_device_status(0)
        assert all(torch.equal(x, y) for x, y in zip(outs, got)) and all(torch.equal(x, y) for x, y in zip(c, plain))
    side = torch.cuda.Stream()
    a = fa.forward_kv4_tree(q, c, lens, table, tree, stream=side)
    side.synchronize()
    b = fa.forward_kv4_tree(q, c, lens, table, tree)
    ok()
    assert torch.equal(a[0], b[0])
