"""Attention of packed sequences with grouped heads: plan, forward, backward, autograd.

Compared with the fp64 reference (oracle/packed.py) within bounds made of the formats:

S    products of bf16 are exact, their fp32 sum of d terms is off by at most 2^-23 of its largest partial sum a term
     (which reach = scale sum |q k| bounds); the product with scale log2 e and the subtraction of the maximum
     round by 2^-24 each: eS = (d + 16) 2^-23 reach.
LSE  its scores' error; the fp32 sum of n terms and the exponential: eS + (n + 64) 2^-23 + 2^-22 (|LSE| + 1).
O    a P is rounded to bf16 (2^-8 of itself) and carries the factor exp(eS) twice (itself and the sum it is divided by); the
     sum of n products is in fp32; the divisor is a sum of rounded or of unrounded P:
     (2^-8 + 2 eS + (n + 64) 2^-22) (sum p |v| + |O|), and bf16's rounding of the result, 2^-8 |O|.
dV   sum P dO with P rounded to bf16: (2^-8 + n 2^-23) sum P |dO|, P's own error eP (S's, and LSE log2 e's product,
     2^-23 |LSE|), and the result's rounding 2^-8 |dV|.
dS   P (dP - D) in fp32, rounded to bf16: its P's eP, the errors of dP and D (sums of d terms), 2^-8 of itself.
dQ, dK  scale sum dS k, scale sum dS q: those errors on the sums of magnitudes, (2^-8 + n 2^-23) sum |dS k|, and 2^-8 |dQ|.
n counts the terms of a sum (for dK and dV the query heads of a key head times the rows).
"""
import ctypes

import numpy as np
import pytest
import torch

import exact_attention_32_gb300 as fa
from oracle import packed as ref

gpu = pytest.mark.gpu
H8 = 2.0 ** -8  # half a step of bf16, relative


def f64(t):
    return t.double().cpu().numpy()


def randn(*shape, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (gain * torch.randn(*shape, generator=g)).bfloat16()


def offsets(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int64)


def batch(lens, H, Hkv, d, seed, first=0, tail=0, gain=1.0):
    cu = offsets(lens, first)
    T = max(1, int(cu[-1]) + tail)
    return (randn(T, H, d, seed=seed, gain=gain), randn(T, Hkv, d, seed=seed + 1), randn(T, Hkv, d, seed=seed + 2), cu)


def dev_cu(cu):
    return torch.tensor(np.asarray(cu), dtype=torch.int32, device="cuda")


def ok():
    torch.cuda.synchronize()
    assert fa.fa_get_device_status(0) == 0


def check_forward(o, lse, q, k, v, cu, scale, causal):
    r = ref.forward(f64(q), f64(k), f64(v), cu, scale, causal)
    d, n = q.shape[2], int(max(np.diff(cu).max(), 1))
    es = (d + 16) * 2.0 ** -23 * r["reach"]
    on = np.isfinite(r["lse"])
    lse, o = f64(lse), f64(o)
    assert (lse[~on] == -np.inf).all() and (o.transpose(1, 0, 2)[~on] == 0).all()
    bound = es + (n + 64) * 2.0 ** -23 + 2.0 ** -22 * (np.abs(r["lse"], where=on, out=np.zeros_like(es)) + 1)
    err = np.abs(np.where(on, lse - np.where(on, r["lse"], 0), 0))
    assert np.isfinite(lse[on]).all() and (err <= bound).all(), (err - bound).max()
    bound = (H8 + 2 * es.T[..., None] + (n + 64) * 2.0 ** -22) * (r["spread"] + np.abs(r["o"])) + H8 * np.abs(r["o"]) + 1e-30
    err = np.abs(o - r["o"])
    assert np.isfinite(o).all() and (err <= bound).all(), (err / bound).max()


def check_backward(got, q, k, v, o, lse, dout, cu, scale, causal):
    r = ref.backward(f64(q), f64(k), f64(v), f64(o), f64(lse), f64(dout), cu, scale, causal)
    d, G = q.shape[2], q.shape[1] // k.shape[1]
    n = int(max(np.diff(cu).max(), 1))
    for name, g in zip(("dq", "dk", "dv"), got):
        terms = n * (1 if name == "dq" else G)
        bound = (H8 + (terms + 16) * 2.0 ** -23) * r[name + "_abs"] + (1 + H8) * (
            r[name + "_p"] + (d + 16) * 2.0 ** -23 * r[name + "_ds"])
        bound = bound * 1.02 + H8 * (np.abs(r[name]) + bound) + 1e-30  # (second order: 2^-8 of 2^-8, and exp(e) - 1 - e)
        g = f64(g)
        err = np.abs(g - r[name])
        assert np.isfinite(g).all() and (err <= bound).all(), (name, (err / bound).max())


# --------------------------------------------------------------------------- the reference (CPU)

def test_reference_forward_is_the_textbook_softmax_of_each_sequence():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((9, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    r = ref.forward(q, k, v, [1, 4, 4, 8], 0.3, True)
    e = np.exp(0.3 * k[4:7, 1] @ q[6, 3])  # row 2 of the third sequence, head 3: key head 1
    assert np.allclose(r["o"][6, 3], e / e.sum() @ v[4:7, 1], atol=1e-14) and np.isclose(r["lse"][3, 6], np.log(e.sum()))
    assert (r["lse"][:, [0, 8]] == -np.inf).all() and (r["o"][[0, 8]] == 0).all()


@pytest.mark.parametrize("causal", [False, True])
def test_reference_gradients_are_the_differences(causal):
    rng = np.random.default_rng(1)
    q, k, v, go = (rng.standard_normal((7, h, 4)) for h in (4, 2, 2, 4))
    cu = [0, 3, 7]
    f = ref.forward(q, k, v, cu, 0.5, causal)
    r = ref.backward(q, k, v, f["o"], f["lse"], go, cu, 0.5, causal)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        num = np.zeros_like(x)
        for i in np.ndindex(x.shape):
            keep = x[i]
            x[i] = keep + 1e-5
            up = (ref.forward(q, k, v, cu, 0.5, causal)["o"] * go).sum()
            x[i] = keep - 1e-5
            num[i] = (up - (ref.forward(q, k, v, cu, 0.5, causal)["o"] * go).sum()) / 2e-5
            x[i] = keep
        # central differences of a smooth function: 1e-10 of the third derivative, and 1e-16 / 1e-5 of rounding
        assert np.abs(num - r[name]).max() < 1e-8


# ------------------------------------------------------------------------------ refusals (CPU)

def _rows(T, heads, d, at, ts=None, hs=None):
    return fa.RowsStruct(at, heads * d if ts is None else ts, d if hs is None else hs)


def _fwd(T=100, B=2, H=4, Hkv=2, d=64, scale=0.1, causal=1, fill=0, **kw):
    r = {n: _rows(T, h, d, 1 << (20 + 4 * i)) for i, (n, h) in enumerate([("q", H), ("k", Hkv), ("v", Hkv), ("o", H)])}
    r.update(kw)
    return fa.fa_fwd_packed(r["q"], r["k"], r["v"], r["o"], 1 << 40, 1 << 41, B, T, H, Hkv, d, scale, causal, fill, 0)


def _bwd(T=100, B=2, H=4, Hkv=2, d=64, scale=0.1, causal=1, fill=0, workspace=1 << 50, **kw):
    names = ["q", "k", "v", "o", "dout", "dq", "dk", "dv"]
    r = {n: _rows(T, Hkv if n in ("k", "v", "dk", "dv") else H, d, 1 << (20 + 2 * i)) for i, n in enumerate(names)}
    r.update(kw)
    return fa.fa_bwd_packed(r["q"], r["k"], r["v"], r["o"], 1 << 45, *(r[n] for n in names[4:]), 1 << 46, B, T, H, Hkv, d, scale,
                            causal, fill, 1 << 47, workspace, 0)


BAD = [dict(T=0), dict(B=0), dict(H=0), dict(Hkv=0), dict(H=5), dict(T=-1), dict(T=1 << 31), dict(B=1 << 31), dict(H=1 << 21, Hkv=1),
       dict(d=0), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(causal=2), dict(fill=2),
       dict(T=1 << 30, H=1 << 10), dict(B=1 << 30, H=4)]


@pytest.mark.parametrize("kw", BAD)
def test_bad_sizes_are_refused_before_any_device_call(kw):
    assert _fwd(**kw) == 1 and _bwd(**kw) == 1


@pytest.mark.parametrize("d", [32, 96, 256])
def test_other_head_dimensions_are_unsupported(d):
    assert _fwd(d=d) == 2 and _bwd(d=d) == 2
    assert fa.fa_bwd_packed_workspace_bytes(1, 1, 1, 1, d) == -1


@pytest.mark.parametrize("ts,hs", [(0, 64), (256, 0), (252, 64), (256, 60), (-256, 64), (1 << 39, 64), (64, 32), (1 << 37, 64)])
def test_bad_strides_are_refused_before_any_device_call(ts, hs):
    for n in ("q", "o"):
        assert _fwd(**{n: _rows(100, 4, 64, 1 << 20, ts, hs)}) == 1
        assert _bwd(**{n: _rows(100, 4, 64, 1 << 20, ts, hs)}) == 1


def test_outputs_whose_rows_meet_are_refused():
    # tokens 128 apart, heads 64 apart: head 2 of a token is head 0 of the next
    assert _fwd(o=_rows(100, 4, 64, 1 << 32, 128, 64)) == 1
    for n in ("dq", "dk", "dv"):
        assert _bwd(**{n: _rows(100, 4, 64, 1 << 32, 64, 64)}) == 1


def test_small_workspace_and_null_tensors_are_refused():
    need = fa.fa_bwd_packed_workspace_bytes(2, 100, 4, 2, 64)
    assert need > 0 and _bwd(workspace=need - 1) == 1
    L = fa.lib()
    assert L.fa_fwd_packed(None, None, None, None, 1 << 40, 1 << 41, 1, 1, 1, 1, 64, 0.1, 0, 0, 0) == 1


def test_plan_sizes():
    for B, T in [(0, 1), (1, 0), (1 << 31, 1), (1, 1 << 31), (-1, 5)]:
        assert fa.fa_packed_plan_bytes(B, T) == -1 and fa.fa_packed_plan(16, B, T, 0, 16, 1 << 40, 0) == 1
    n = fa.fa_packed_plan_bytes(3, 1000)
    # a header, an entry of 16 bytes for each block of 128 and of 256 rows that the lengths could make, one a sequence
    assert n == 128 + 16 * (1000 // 128 + 3 + 1000 // 256 + 3 + 3)
    assert fa.fa_packed_plan(16, 3, 1000, 0, 16, n - 1, 0) == 1 and fa.fa_packed_plan(16, 3, 1000, 2, 16, n, 0) == 1


def test_the_largest_number_of_sequences():
    # the plan goes 1024 of them at a time, and the number behind the last ones has to fit 31 bits
    most = (1 << 31) - 2048
    assert fa.fa_packed_plan_bytes(most, 1) == 128 + 16 * 3 * most
    for B in (most + 1, (1 << 31) - 1024, (1 << 31) - 1023, (1 << 31) - 512):
        assert fa.fa_packed_plan_bytes(B, 1) == -1 and fa.fa_packed_plan(16, B, 1, 0, 16, 1 << 50, 0) == 1
        assert fa.fa_bwd_packed_workspace_bytes(B, 1, 1, 1, 64) == -1
    assert fa.fa_packed_plan_bytes(1, (1 << 31) - 512) > 0 and fa.fa_packed_plan_bytes(1, (1 << 31) - 511) == -1


def test_python_calls_refuse_wrong_tensors():
    q, k, cu = torch.zeros(4, 2, 64).bfloat16(), torch.zeros(4, 1, 64).bfloat16(), torch.zeros(2, dtype=torch.int32)
    for bad in (lambda: fa.forward_packed(q, k, k, cu), lambda: fa.forward_packed(1, k, k, cu), lambda: fa.packed_plan(cu, 4),
                lambda: fa.backward_packed(q, k, k, q, q, q, cu), lambda: fa.attention_packed(q, k, k, cu)):
        with pytest.raises(ValueError):
            bad()


# --------------------------------------------------------------------------------- forward (GPU)

LENS = [[1], [2], [127], [128], [129], [255, 1], [256], [257], [17, 0, 120, 1], [300, 5, 0, 0, 64, 128, 1], [0, 0, 3], [700, 33]]


@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 64), (4, 1, 128), (6, 2, 64), (3, 3, 128), (8, 4, 64)])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_forward_over_short_and_odd_lengths(lens, H, Hkv, d, causal):
    q, k, v, cu = batch(lens, H, Hkv, d, seed=sum(lens) + H)
    o, lse = fa.forward_packed(q.cuda(), k.cuda(), v.cuda(), dev_cu(cu), causal=causal)
    ok()
    check_forward(o, lse, q, k, v, cu, fa.default_scale(d), causal)


@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,H,Hkv,d,gain", [([1500, 1, 900, 77], 4, 2, 128, 1.0), ([2048, 130], 3, 1, 64, 8.0),
                                              ([1000] * 5, 2, 2, 128, 8.0), ([40] * 90, 8, 2, 64, 1.0),
                                              # few long items, which clusters of 2 to 4 share; short sequences beside them
                                              ([3000], 4, 2, 128, 1.0), ([2900, 1, 3300], 2, 1, 64, 4.0), ([3, 4100], 1, 1, 128, 8.0),
                                              ([4500, 129], 2, 2, 64, 1.0), ([2700], 3, 1, 128, 1.0)])
def test_forward_over_many_tiles_and_large_scores(lens, H, Hkv, d, gain, causal):
    q, k, v, cu = batch(lens, H, Hkv, d, seed=5, gain=gain)
    o, lse = fa.forward_packed(q.cuda(), k.cuda(), v.cuda(), dev_cu(cu), causal=causal)
    ok()
    check_forward(o, lse, q, k, v, cu, fa.default_scale(d), causal)


@gpu
@pytest.mark.parametrize("lens,H,Hkv", [([4, 600, 1], 4, 2), ([4, 600, 1], 3, 3), ([9000], 1, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [-2.0 ** 29, -3e6, 3e6, 2.0 ** 29])
def test_scores_up_to_two_to_the_twenty_ninth(size, d, lens, H, Hkv):
    # all queries alike, keys 1, 1, 4 and 4 (a quarter of the rows each) in every channel: those of the largest score tie, the others weigh
    # nothing.  O is their mean: P's rounding (bf16, 2^-8, which the divisor may not share) and the result's
    T, scale = sum(lens), fa.default_scale(d)
    cu = offsets(lens)
    key = np.concatenate([np.array([1.0, 1.0, 4.0, 4.0])[np.arange(n) * 4 // n] for n in lens])
    top = 4 if size > 0 else 1
    k = torch.tensor(key).bfloat16()[:, None, None].expand(T, Hkv, d).contiguous()
    q, v = torch.full((T, H, d), size / (top * d * scale)).bfloat16(), randn(T, Hkv, d, seed=61)
    o, lse = fa.forward_packed(q.cuda(), k.cuda(), v.cuda(), dev_cu(cu))
    ok()
    for a, e in zip(cu[:-1], cu[1:]):
        s = float(q[0, 0, 0]) * scale * d * key[a:e]
        tie = s == s.max()
        want = f64(v[a:e])[tie].mean(0).repeat(H // Hkv, 0)
        spread = np.abs(f64(v[a:e])[tie]).mean(0).repeat(H // Hkv, 0)
        want_lse = s.max() + np.log(tie.sum())
        assert (np.abs(f64(lse)[:, a:e] - want_lse) <= (d + 16) * 2.0 ** -23 * abs(want_lse)).all()
        bound = (H8 + (e - a + 64) * 2.0 ** -22) * (spread + np.abs(want)) + H8 * np.abs(want)
        assert (np.abs(f64(o)[a:e] - want) <= bound).all()


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_one_sequence_of_equal_heads_is_the_dense_forward(d):
    q, k, v = (t.cuda() for t in fa.make_inputs(1, 3, 1111, d, seed=9))
    o, lse = fa.forward(q, k, v, causal=True)
    head_major = [t[0].transpose(0, 1) for t in (q, k, v)]  # [T, H, d] with heads outermost in memory
    got, got_lse = fa.forward_packed(*head_major, dev_cu([0, 1111]), causal=True)
    ok()
    # two roundings of one value, each off by P's 2^-8 and the output's 2^-8 of sum p |v|, which |v| bounds
    top = v.float().abs().max().item()
    assert (got.float() - o[0].transpose(0, 1).float()).abs().max().item() <= 4 * H8 * top
    assert (got_lse - lse[0]).abs().max().item() <= 1e-4


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 2), (3, 3)])
def test_slices_of_one_projection_and_given_outputs(H, Hkv, d):
    lens = [130, 1, 64, 301]
    cu = offsets(lens, first=3)
    T = int(cu[-1]) + 9
    qkv = randn(T, H + 2 * Hkv, d, seed=11)
    g = qkv.cuda()
    q, k, v = g[:, :H], g[:, H:H + Hkv], g[:, H + Hkv:]
    wide = torch.full((T, H + 1, d + 8), 7.0, device="cuda").bfloat16()
    out, lse = wide[:, :H, :d], torch.full((H, T), 5.0, device="cuda")
    for causal in (False, True):
        fa.forward_packed(q, k, v, dev_cu(cu), causal=causal, out=out, lse=lse)
        ok()
        # rows of no sequence, and what lies between the rows, are as they were
        assert (wide[:, H:] == 7).all() and (wide[:, :, d:] == 7).all() and (out[:3] == 7).all() and (out[cu[-1]:] == 7).all()
        assert (lse[:, :3] == 5).all() and (lse[:, cu[-1]:] == 5).all()
        o, l = out.clone(), lse.clone()
        o[:3], o[cu[-1]:], l[:, :3], l[:, cu[-1]:] = 0, 0, -np.inf, -np.inf
        check_forward(o, l, qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:], cu, fa.default_scale(d), causal)
        o2, l2 = fa.forward_packed(q, k, v, dev_cu(cu), causal=causal)  # tensors of its own: filled
        ok()
        assert torch.equal(o2, o) and torch.equal(l2, l)
    o3, l3 = fa.forward_packed(q, k, v, dev_cu(cu), causal=True, out=torch.empty_like(o))  # one given: the other filled
    o4, l4 = fa.forward_packed(q, k, v, dev_cu(cu), causal=True, lse=torch.empty_like(l))
    ok()
    assert torch.equal(l3, l) and torch.equal(o4, o) and torch.equal(o3[3:cu[-1]], o[3:cu[-1]])
    assert torch.equal(l4[:, 3:cu[-1]], l[:, 3:cu[-1]])


@gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("H,Hkv,d,last", [(4, 2, 64, 150), (2, 2, 128, 150), (4, 1, 128, 150), (3, 1, 64, 150), (2, 1, 128, 9000), (1, 1, 64, 9000)])
def test_what_other_sequences_hold_stays_out(H, Hkv, d, last, causal, value):
    # the second of three sequences, and the rows behind the last, hold rubbish; the others are as without it
    lens = [77, 100, last]
    q, k, v, cu = batch(lens, H, Hkv, d, seed=21, tail=60)
    dout = randn(*q.shape, seed=24)
    bad = [t.clone() for t in (q, k, v, dout)]
    for t in bad:
        t[77:177] = value
        t[cu[-1]:] = value
    res = []
    for x in ((q, k, v, dout), bad):
        a = [t.cuda() for t in x]
        o, lse = fa.forward_packed(*a[:3], dev_cu(cu), causal=causal)
        res.append((o, lse.T, *fa.backward_packed(*a[:3], o, lse, a[3], dev_cu(cu), causal=causal)))
    ok()
    keep = torch.cat([torch.arange(77), torch.arange(177, len(q))])
    for i, (x, y) in enumerate(zip(*res)):
        if i == 2:  # dQ's parts meet in no fixed order: bf16's two nearest values of one sum
            assert torch.isfinite(y[keep]).all()
            assert ((x[keep].float() - y[keep].float()).abs() <= 2 * H8 * x[keep].float().abs() + 1e-5).all()
        else:
            assert torch.equal(x[keep], y[keep])


@gpu
def test_a_value_that_is_not_finite_reaches_no_earlier_block_of_its_sequence():
    q, k, v, cu = batch([400, 50], 4, 2, 128, seed=31)
    v[300] = float("nan")  # the third block of 128
    o, _ = fa.forward_packed(q.cuda(), k.cuda(), v.cuda(), dev_cu(cu), causal=True)
    k[300], v[300] = float("nan"), 1.0
    o2, _ = fa.forward_packed(q.cuda(), k.cuda(), v.cuda(), dev_cu(cu), causal=True)
    ok()
    assert torch.isfinite(o[:256]).all() and torch.isfinite(o[400:]).all() and torch.isnan(o[300:400]).all()
    assert torch.isfinite(o2[:300]).all() and torch.isfinite(o2[400:]).all()  # a key's scores are masked one by one


@gpu
def test_plan_made_ahead_and_used_for_several_layers():
    lens = [200, 3, 511]
    cu = offsets(lens)
    plan = fa.packed_plan(dev_cu(cu), int(cu[-1]), causal=True)
    for seed in (41, 42):
        q, k, v, _ = batch(lens, 4, 2, 64, seed=seed)
        a = [t.cuda() for t in (q, k, v)]
        o, lse = fa.forward_packed(*a, dev_cu(cu), causal=True, plan=plan)
        o2, lse2 = fa.forward_packed(*a, dev_cu(cu), causal=True)
        ok()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for bad in (dict(causal=False), dict(plan=plan._replace(tokens=3)), dict(plan=plan._replace(sequences=1)), dict(plan=(1, 2))):
        with pytest.raises(ValueError):
            fa.forward_packed(*a, dev_cu(cu), **{"causal": True, "plan": plan, **bad})


@gpu
def test_a_plan_of_another_batch_does_nothing_and_is_reported():
    q, k, v, cu = batch([100, 28], 2, 2, 64, seed=51)
    a = [t.cuda() for t in (q, k, v)]
    other = fa.packed_plan(dev_cu([0, 50, 64]), 64, causal=True)  # fewer rows; its memory would serve
    need = fa.fa_packed_plan_bytes(2, 128)
    table = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for t in (table, torch.cat([other.table, table])[:need].contiguous()):
        out, lse = torch.full_like(a[0], 3.0), torch.full((2, 128), 3.0, device="cuda")
        fa.forward_packed(*a, dev_cu(cu), causal=True, plan=fa.PackedPlan(t, 128, 2, True), out=out, lse=lse)
        torch.cuda.synchronize()
        assert fa.fa_get_device_status(0) == 9 and (out == 3).all() and (lse == 3).all()
        grads = tuple(torch.full_like(x, 3.0) for x in a)
        fa.backward_packed(*a, out, lse, a[0], dev_cu(cu), causal=True, plan=fa.PackedPlan(t, 128, 2, True), out=grads)
        torch.cuda.synchronize()
        assert fa.fa_get_device_status(0) == 9 and all((g == 3).all() for g in grads)
    fa.forward_packed(*a, dev_cu(cu), causal=True)
    ok()


@gpu
def test_a_plan_holds_its_own_offsets():
    # of the same number of sequences and rows: the plan's lengths are what counts, as its documentation says, in both directions
    q, k, v, cu = batch([100, 28], 4, 2, 64, seed=53)
    a, other = [t.cuda() for t in (q, k, v)], [0, 30, 128]
    plan = fa.packed_plan(dev_cu(other), 128, causal=True)
    o, lse = fa.forward_packed(*a, dev_cu(cu), causal=True, plan=plan)
    want = fa.forward_packed(*a, dev_cu(other), causal=True)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    check_forward(o.cpu(), lse.cpu(), q, k, v, np.array(other), fa.default_scale(64), True)
    got = fa.backward_packed(*a, o, lse, a[0], dev_cu(cu), causal=True, plan=plan)
    ok()
    check_backward(got, q, k, v, o, lse, q, np.array(other), fa.default_scale(64), True)


@gpu
@pytest.mark.parametrize("cu,held", [([0, 50, 40, 100], [0, 50, 50, 100]), ([-5, 30, 60, 90], [0, 30, 60, 90]),
                                     ([0, 30, 60, 500], [0, 30, 60, 100]), ([0, 2 ** 31 - 1, 60, 100], [0, 100, 100, 100]),
                                     ([200, 300, -300, 5], [100, 100, 100, 100])])
def test_offsets_that_do_not_ascend_are_held_and_reported(cu, held):
    q, k, v, _ = batch([100], 4, 2, 64, seed=61)
    o, lse = fa.forward_packed(q.cuda(), k.cuda(), v.cuda(), dev_cu(cu), causal=True)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status(0) == 9
    check_forward(o, lse, q, k, v, np.array(held), fa.default_scale(64), True)
    ok()


def plan_lists(plan):
    raw = plan.table.cpu().numpy().view(np.int32)
    head, T, B = raw[:8], plan.tokens, plan.sequences
    e = raw[32:].reshape(-1, 4)
    return head, e[:T // 128 + B][:head[4]], e[T // 128 + B:T // 128 + B + T // 256 + B][:head[5]]


@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [[1], [0, 5, 0], [300, 128, 129, 1], list(range(1, 2600, 7)), [140000, 3, 270000], [0] * 2100 + [130] + [1] * 1500])
def test_plan_names_every_block_once_the_longest_loops_first(lens, causal):
    cu = offsets(lens, first=2)
    plan = fa.packed_plan(dev_cu(cu), int(cu[-1]) + 3, causal=causal)
    ok()
    head, blocks, pairs = plan_lists(plan)
    assert head[1] == cu[-1] + 3 and head[2] == len(lens) and head[6] == 2 and head[7] == cu[-1]
    n = -(-np.asarray(lens) // 128)
    first = np.concatenate([[0], np.cumsum(n)])
    for got, rows in ((blocks, 128), (pairs, 256)):
        want = [(a, m, i, f) for a, m, f in zip(cu, lens, first) for i in range(-(-m // rows))]
        assert sorted(map(tuple, got.tolist())) == sorted(map(tuple, np.array(want).reshape(-1, 4).tolist()))
        tiles = -(-got[:, 1] // 128)
        loop = np.minimum(tiles, (got[:, 2] + 1) * (rows // 128)) if causal else tiles
        shift = max(0, int(n.max()).bit_length() - 10)
        assert (np.diff(loop >> shift) <= 0).all()


# -------------------------------------------------------------------------------- backward (GPU)

@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 64), (4, 1, 128), (6, 2, 64), (3, 3, 128), (8, 4, 64)])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_backward_over_short_and_odd_lengths(lens, H, Hkv, d, causal):
    q, k, v, cu = batch(lens, H, Hkv, d, seed=sum(lens) + H + 100)
    dout, scale = randn(*q.shape, seed=7), fa.default_scale(d)
    a = [t.cuda() for t in (q, k, v)]
    o, lse = fa.forward_packed(*a, dev_cu(cu), causal=causal)
    got = fa.backward_packed(*a, o, lse, dout.cuda(), dev_cu(cu), causal=causal)
    ok()
    check_backward(got, q, k, v, o, lse, dout, cu, scale, causal)


@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,H,Hkv,d,gain", [([1500, 1, 900, 77], 4, 2, 128, 1.0), ([1100, 130], 3, 1, 64, 4.0),
                                              ([600] * 4, 2, 2, 128, 4.0), ([40] * 90, 8, 2, 64, 1.0), ([700], 16, 1, 128, 1.0),
                                              (list(range(1, 300, 9)), 16, 8, 128, 1.0), (list(range(1, 300, 9)), 8, 8, 64, 1.0),
                                              ([1500, 1, 1, 2], 2, 1, 64, 1.0), ([1030], 4, 1, 128, 1.0), ([900, 17], 3, 1, 128, 1.0)])
def test_backward_over_many_tiles_and_large_scores(lens, H, Hkv, d, gain, causal):
    q, k, v, cu = batch(lens, H, Hkv, d, seed=15, gain=gain)
    dout, scale = randn(*q.shape, seed=8), fa.default_scale(d)
    a = [t.cuda() for t in (q, k, v)]
    o, lse = fa.forward_packed(*a, dev_cu(cu), causal=causal)
    got = fa.backward_packed(*a, o, lse, dout.cuda(), dev_cu(cu), causal=causal)
    again = fa.backward_packed(*a, o, lse, dout.cuda(), dev_cu(cu), causal=causal)
    ok()
    check_backward(got, q, k, v, o, lse, dout, cu, scale, causal)
    assert torch.equal(got[1], again[1]) and torch.equal(got[2], again[2])  # (dQ's parts meet in no fixed order)


@gpu
@pytest.mark.parametrize("H,Hkv,d", [(4, 2, 64), (3, 3, 128), (8, 1, 128)])
def test_gradients_into_slices_of_one_gradient(H, Hkv, d):
    lens = [130, 1, 64, 301]
    cu = offsets(lens, first=3)
    T = int(cu[-1]) + 9
    qkv, dout = randn(T, H + 2 * Hkv, d, seed=12), randn(T, H, d, seed=13)
    g = qkv.cuda()
    q, k, v = g[:, :H], g[:, H:H + Hkv], g[:, H + Hkv:]
    o, lse = fa.forward_packed(q, k, v, dev_cu(cu), causal=True)
    grad = torch.full_like(g, 7.0)
    out = grad[:, :H], grad[:, H:H + Hkv], grad[:, H + Hkv:]
    got = fa.backward_packed(q, k, v, o, lse, dout.cuda(), dev_cu(cu), causal=True, out=out)
    own = fa.backward_packed(q, k, v, o, lse, dout.cuda(), dev_cu(cu), causal=True)
    ok()
    assert (grad[:3] == 7).all() and (grad[cu[-1]:] == 7).all() and all(x.data_ptr() == y.data_ptr() for x, y in zip(got, out))
    for x in own:
        assert (x[:3] == 0).all() and (x[cu[-1]:] == 0).all()
    grad[:3], grad[cu[-1]:] = 0, 0
    parts = [qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]]
    check_backward(out, *parts, o, lse, dout, cu, fa.default_scale(d), True)
    check_backward(own, *parts, o, lse, dout, cu, fa.default_scale(d), True)


@gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("H,Hkv,d", [(4, 2, 64), (3, 3, 128), (8, 1, 128), (1, 1, 64)])
def test_head_major_tensors_and_gradients(H, Hkv, d, causal):
    # [heads, T, d] in memory, each head's rows in a longer run of them; gradients and O into such tensors too
    lens = [130, 1, 64, 0, 301]
    cu = offsets(lens, first=3)
    T = int(cu[-1]) + 9

    def head_major(t):  # [T, heads, d] -> the same, heads outermost with 5 rows of 7 between them
        wide = torch.full((t.shape[1], T + 5, d), 7.0, device="cuda").bfloat16()
        wide[:, :T] = t.cuda().transpose(0, 1)
        return wide, wide[:, :T].transpose(0, 1)

    cpu = [randn(T, h, d, seed=31 + i) for i, h in enumerate((H, Hkv, Hkv, H))]
    q, k, v, dout = (head_major(t)[1] for t in cpu)
    seven = [head_major(torch.full_like(t, 7.0)) for t in (cpu[0], *cpu[:3])]
    o, *grads = (view for _, view in seven)
    lse = torch.full((H, T), 7.0, device="cuda")
    fa.forward_packed(q, k, v, dev_cu(cu), causal=causal, out=o, lse=lse)
    fa.backward_packed(q, k, v, o, lse, dout, dev_cu(cu), causal=causal, out=grads)
    ok()
    outside = [0, 1, 2, *range(int(cu[-1]), T)]
    for (wide, view) in seven:
        assert (wide[:, T:] == 7).all() and (view[outside] == 7).all()
        view[outside] = 0
    assert (lse[:, outside] == 7).all()
    lse[:, outside] = -np.inf
    check_forward(o, lse, *cpu[:3], cu, fa.default_scale(d), causal)
    check_backward(grads, *cpu[:3], o, lse, cpu[3], cu, fa.default_scale(d), causal)


@gpu
@pytest.mark.parametrize("d,causal", [(64, True), (128, False)])
def test_autograd_of_packed_attention(d, causal):
    q, k, v, cu = batch([90, 0, 200, 7], 4, 2, d, seed=71, first=1, tail=2)
    dout, scale = randn(*q.shape, seed=74), fa.default_scale(d)
    a = [t.cuda().requires_grad_(True) for t in (q, k, v)]
    plan = fa.packed_plan(dev_cu(cu), len(q), causal=causal)
    for p in (None, plan):
        for t in a:
            t.grad = None
        o = fa.attention_packed(*a, dev_cu(cu), causal=causal, plan=p)
        o.backward(dout.cuda())
        ok()
        lse = fa.forward_packed(*(t.detach() for t in a), dev_cu(cu), causal=causal)[1]
        check_backward([t.grad for t in a], q, k, v, o.detach(), lse, dout, cu, scale, causal)
    # a gradient that is broadcast (a sum's) and inputs that are slices
    qkv = torch.cat([q, k, v], 1).cuda().requires_grad_(True)
    o = fa.attention_packed(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], dev_cu(cu), causal=causal)
    o.sum().backward()
    ok()
    lse = fa.forward_packed(*(t.detach() for t in a), dev_cu(cu), causal=causal)[1]
    g = qkv.grad
    check_backward((g[:, :4], g[:, 4:6], g[:, 6:]), q, k, v, o.detach(), lse, torch.ones_like(dout), cu, scale, causal)


# ------------------------------------------------------------------------ streams, graphs, refusals (GPU)

@gpu
def test_captured_step_replays_with_new_lengths():
    H, Hkv, d, T = 4, 2, 64, 400
    q, k, v, _ = batch([T], H, Hkv, d, seed=81)
    dout = randn(T, H, d, seed=84)
    a = [t.cuda() for t in (q, k, v, dout)]
    cu = dev_cu([0, 100, 400])
    fa.forward_packed(*a[:3], cu, causal=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = fa.packed_plan(cu, T, causal=True)
        o, lse = fa.forward_packed(*a[:3], cu, causal=True, plan=plan)
        grads = fa.backward_packed(*a[:3], o, lse, a[3], cu, causal=True, plan=plan)
    for offs in ([0, 100, 400], [0, 399, 400], [7, 7, 300]):
        cu.copy_(torch.tensor(offs, dtype=torch.int32))
        graph.replay()
        ok()
        check_forward(o, lse, q, k, v, np.array(offs), fa.default_scale(d), True)
        check_backward(grads, q, k, v, o, lse, dout, np.array(offs), fa.default_scale(d), True)


@gpu
def test_calls_on_several_streams_at_once():
    sets = []
    for i, (lens, H, Hkv, d, causal) in enumerate([([500, 40], 4, 2, 64, True), ([300, 301], 2, 2, 128, False), ([64] * 9, 8, 1, 64, True)]):
        q, k, v, cu = batch(lens, H, Hkv, d, seed=90 + i)
        a = [t.cuda() for t in (q, k, v, randn(*q.shape, seed=95 + i))]
        sets.append((a, dev_cu(cu), causal))

    def run(a, cu, causal, stream=None):
        o, lse = fa.forward_packed(*a[:3], cu, causal=causal, stream=stream)
        return o, lse, *fa.backward_packed(*a[:3], o, lse, a[3], cu, causal=causal, stream=stream)[1:]
    alone = [run(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [run(*s, stream=st) for s, st in zip(sets, streams)]
        ok()
        for x, y in zip(alone, got):
            assert all(torch.equal(p, r) for p, r in zip(x, y))


@gpu
def test_calls_from_threads_that_have_made_no_other():
    # each call the first of its thread, which has no context then (as autograd's threads do not)
    import threading
    q, k, v, cu = batch([40, 60], 4, 2, 64, seed=97)
    a = [t.cuda() for t in (q, k, v)]
    c = dev_cu(cu)
    o, lse = fa.forward_packed(*a, c)
    dense = [t.transpose(0, 1)[None].contiguous() for t in (a[0], a[0], a[0])]
    cache, lens, table = fa.kv4_cache(4, 2, 16, 64), torch.tensor([20]).int().cuda(), torch.tensor([[0, 1]]).int().cuda()
    got, errors = {}, []
    ok()

    def run(name, f):
        try:
            got[name] = f()
        except Exception as e:  # noqa: BLE001
            errors.append((name, e))
    calls = dict(fwd=lambda: fa.forward_packed(*a, c), bwd=lambda: fa.backward_packed(*a, o, lse, o, c), dense=lambda: fa.forward(*dense),
                 kv4=lambda: fa.forward_kv4(a[0][None, :1].transpose(1, 2).contiguous(), cache, lens, table),
                 weights=lambda: fa.key_weights(dense[0], dense[0], torch.zeros(1, 4, 100, device="cuda")))
    for name, f in calls.items():
        t = threading.Thread(target=run, args=(name, f))
        t.start()
        t.join()
    ok()
    assert not errors and torch.equal(got["fwd"][0], o) and len(got) == len(calls)


@gpu
def test_python_calls_refuse_wrong_gpu_tensors():
    q, k, v, cu = batch([40, 60], 4, 2, 64, seed=99)
    a = [t.cuda() for t in (q, k, v)]
    c = dev_cu(cu)
    o, lse = fa.forward_packed(*a, c)
    bad = [lambda: fa.forward_packed(a[0].float(), *a[1:], c), lambda: fa.forward_packed(a[0], a[1][:50], a[2], c),
           lambda: fa.forward_packed(a[0][:, :3], *a[1:], c), lambda: fa.forward_packed(a[0][:, :1].expand(-1, 4, -1), *a[1:], c),
           lambda: fa.forward_packed(a[0].transpose(1, 2), *a[1:], c), lambda: fa.forward_packed(*a, c.long()),
           lambda: fa.forward_packed(*a, c[:1]), lambda: fa.forward_packed(*a, c.cpu()), lambda: fa.forward_packed(*a, c, out=a[0][:50]),
           lambda: fa.forward_packed(*a, c, lse=lse.T), lambda: fa.forward_packed(*(t.cpu() for t in a), c),
           lambda: fa.backward_packed(*a, o, lse[:, :50], o, c), lambda: fa.backward_packed(*a, o, lse, o.float(), c),
           lambda: fa.backward_packed(*a, o, lse, o, c, out=(o, o)), lambda: fa.backward_packed(*a, o, lse, o, c, workspace=o)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: fa.forward_packed(*a, c, out=a[0]), lambda: fa.forward_packed(*a, c, scale=0.0),
              lambda: fa.backward_packed(*a, o, lse, o, c, out=(o, a[1], a[2])),
              lambda: fa.backward_packed(*a, o, lse, o, c, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
              lambda: fa.forward_packed(*(t[..., :32] for t in a), c)):
        with pytest.raises(fa.FAError):
            f()
    ok()
    # slices of one buffer that interleave are not one another; the same slice twice is
    n = torch.empty(100, 8, 64, device="cuda").bfloat16()
    fa.backward_packed(*a, o, lse, o, c, out=(n[:, :4], n[:, 4:6], n[:, 6:]))
    for out in ((n[:, :4], n[:, 3:5], n[:, 6:]), (n[:, :4], n[:, 4:6], n[:, 4:6]), (n[:, 4:], n[:, :2], n[:, 6:])):
        with pytest.raises(fa.FAError):
            fa.backward_packed(*a, o, lse, o, c, out=out)
    ok()


@gpu
def test_workspace_is_all_that_is_used():
    q, k, v, cu = batch([129, 64, 1], 4, 2, 64, seed=101)
    a = [t.cuda() for t in (q, k, v)]
    need = fa.fa_bwd_packed_workspace_bytes(3, 194, 4, 2, 64)
    ws = torch.full((need + 1024,), 171, dtype=torch.uint8, device="cuda")
    o, lse = fa.forward_packed(*a, dev_cu(cu))
    got = fa.backward_packed(*a, o, lse, o, dev_cu(cu), workspace=ws[:need])
    ok()
    assert (ws[need:] == 171).all()
    check_backward(got, q, k, v, o, lse, o.cpu(), cu, fa.default_scale(64), False)


@gpu
def test_rows_past_four_gibibytes():
    # 2^31 elements and more between the first row and the last: offsets in elements and bytes pass 32 bits
    T, H, d = 600000, 32, 128
    q = torch.empty(T, H, d, device="cuda", dtype=torch.bfloat16).normal_()
    k = torch.empty(T, 8, d, device="cuda", dtype=torch.bfloat16).normal_()
    cu = [0, 70, T - 300, T - 200, T]  # the long middle is made of no queries that are checked, and skipped as rows of none
    cu = [T - 300, T - 200, T - 1, T]
    out = torch.zeros_like(q)
    lse = torch.zeros(H, T, device="cuda")
    fa.forward_packed(q, k, k, dev_cu(cu), causal=True, out=out, lse=lse)
    ok()
    s = slice(T - 300, T)
    check_forward(out[s].cpu(), lse[:, s].cpu(), q[s].cpu(), k[s].cpu(), k[s].cpu(), np.array(cu) - (T - 300), fa.default_scale(d), True)
    assert (out[:T - 300] == 0).all()


@gpu
def test_gradients_past_four_gibibytes():
    # 2^31 elements and more in q's gradient and in the fp32 accumulator behind it
    H, Hkv, d = 32, 8, 128
    cu = offsets([500] * 1079 + [300, 1, 129])
    T = int(cu[-1])
    q, dout = (torch.empty(T, H, d, device="cuda", dtype=torch.bfloat16).normal_() for _ in range(2))
    k, v = (torch.empty(T, Hkv, d, device="cuda", dtype=torch.bfloat16).normal_() for _ in range(2))
    plan = fa.packed_plan(dev_cu(cu), T, causal=True)
    o, lse = fa.forward_packed(q, k, v, dev_cu(cu), causal=True, plan=plan)
    got = fa.backward_packed(q, k, v, o, lse, dout, dev_cu(cu), causal=True, plan=plan)
    ok()
    middle = (1 << 31) // (H * d) // 500  # the sequence in which element 2^31 lies
    assert cu[middle] * H * d < 1 << 31 < cu[middle + 1] * H * d
    for i in (0, middle, 1079, 1080, 1081):
        s = slice(int(cu[i]), int(cu[i + 1]))
        a = [t[s].cpu() for t in (q, k, v, o, dout)]
        own = np.array([0, s.stop - s.start])
        check_forward(a[3], lse[:, s].cpu(), *a[:3], own, fa.default_scale(d), True)
        check_backward([g[s].cpu() for g in got], *a[:4], lse[:, s].cpu(), a[4], own, fa.default_scale(d), True)
