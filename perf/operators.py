"""The 4-bit KV cache operators, as they are measured: sizes, inputs, their plain
form in elementary torch operations, the framework's calls and the definition in
64 bits.

Kinds of case (a token-head is one token of one key head):
  weights   accumulated attention weight of a prompt's keys from q, k and the forward's LSE
  append    new tokens quantised into the paged cache, then read back as the values they stand for
  read      a range of the cache as bf16 K and V (what a chunked prefill attends to)
  decode    attention of the newest tokens of each sequence over its cache
  evict     the heaviest and the most recent tokens moved to fresh pages, then read back

Cache layout: pages of P tokens, [n_pages, Hkv, P, ...]; E2M1 codes two a byte (the even
channel in the low nibble), one scale byte per 32 channels of K and one per token of V;
a scale byte is the upper magnitude bits of a half (half(byte << 7)).
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one short sequence in one head: the call's latency
        dict(name="weights_n256", kind="weights", B=1, H=1, Hkv=1, N=256, d=64, causal=False, first=0),
        # the benchmark's long causal prompt, every head with its own keys
        dict(name="weights_n16384", kind="weights", B=1, H=32, Hkv=32, N=16384, d=128, causal=True, first=0),
        # a batch's next token each, at lengths that differ
        dict(name="append_token", kind="append", B=64, Hkv=8, S=1, d=128, P=64, longest=2048, weights=True),
        # prompts of different lengths enter the cache with their weights
        dict(name="append_prompts", kind="append", B=8, Hkv=8, S=4096, d=128, P=64, longest=4096, weights=True),
        # a short odd range of small heads
        dict(name="read_short", kind="read", B=3, Hkv=4, T=333, d=64, P=16, longest=1000),
        # the prefix of a long chunked prefill
        dict(name="read_prefix", kind="read", B=4, Hkv=8, T=16384, d=128, P=64, longest=16384),
        # one short conversation: latency
        dict(name="decode_one_short", kind="decode", B=1, H=16, Hkv=4, n_q=1, d=64, P=16, longest=300, ragged=False,
             accumulate=False),
        # one long document: few rows, the long axis has to be split
        dict(name="decode_one_long", kind="decode", B=1, H=32, Hkv=8, n_q=1, d=128, P=64, longest=131072,
             ragged=False, accumulate=False),
        # sequences of very different lengths, three proposed tokens each, weights accumulated for eviction
        dict(name="decode_ragged_weights", kind="decode", B=24, H=32, Hkv=8, n_q=3, d=128, P=32, longest=8192,
             ragged=True, accumulate=True),
        # a full serving batch
        dict(name="decode_batch", kind="decode", B=64, H=64, Hkv=8, n_q=1, d=128, P=64, longest=16384, ragged=False,
             accumulate=False),
        # a small cache over its budget by a few tokens
        dict(name="evict_short", kind="evict", B=4, Hkv=8, d=64, P=16, longest=600, keep=512, recent=64),
        # long prompts cut to a quarter
        dict(name="evict_long", kind="evict", B=16, Hkv=8, d=128, P=64, longest=16384, keep=4096, recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["weights", "append", "read", "decode", "decode", "evict"])
    d, P, Hkv = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 4, 5, 8])
    if kind == "weights":
        N, G = _log(rng, 64, 12000), rng.choice([1, 2, 4, 7, 8])
        # at most the longest listed prompt's products
        B = max(1, min(rng.choice([1, 2, 4]), int(32 * 16384 ** 2 / (N * N * Hkv * G))))
        while Hkv > 1 and B * Hkv * G * N * N > 32 * 16384 ** 2:
            Hkv -= 1
        return dict(kind=kind, B=B, H=Hkv * G, Hkv=Hkv, N=N, d=d, causal=rng.random() < 0.7,
                    first=rng.choice([0, 0, N // 2, N - 1]))
    if kind == "append":
        S, B = _log(rng, 1, 4096), _log(rng, 1, 128)
        B = max(1, min(B, 8 * 4096 // S))
        return dict(kind=kind, B=B, Hkv=Hkv, S=S, d=d, P=P, longest=S + _log(rng, 1, 3000), weights=rng.random() < 0.5)
    if kind == "read":
        T, B = _log(rng, 1, 16384), _log(rng, 1, 32)
        B = max(1, min(B, 4 * 16384 // T))
        return dict(kind=kind, B=B, Hkv=Hkv, T=T, d=d, P=P, longest=T + _log(rng, 1, 500))
    if kind == "decode":
        G, n_q = rng.choice([1, 2, 3, 4, 7, 8, 16]), rng.choice([1, 1, 1, 2, 5, 8])
        longest = max(n_q, _log(rng, 8, 65536))
        B = max(1, min(_log(rng, 1, 96), 64 * 16384 // longest // max(1, G * n_q // 8)))
        return dict(kind=kind, B=B, H=Hkv * G, Hkv=Hkv, n_q=n_q, d=d, P=P, longest=longest, ragged=rng.random() < 0.6,
                    accumulate=rng.random() < 0.4)
    longest = _log(rng, 32, 16384)
    keep = max(1, int(longest * rng.uniform(0.2, 0.9)))
    B = max(1, min(_log(rng, 1, 32), 16 * 16384 // longest))
    return dict(kind=kind, B=B, Hkv=Hkv, d=d, P=P, longest=longest, keep=keep, recent=int(keep * rng.uniform(0, 0.9)))


# ----------------------------------------------------------------- the inputs

def _lengths(g, B, lo, hi, ragged=True):
    """B lengths in [lo, hi], the first of them hi (all of them where not ragged)."""
    n = torch.full((B,), hi, dtype=torch.int32, device="cuda")
    if ragged and B > 1:
        n[1:] = torch.randint(lo, hi + 1, (B - 1,), generator=g, device="cuda", dtype=torch.int32)
    return n


def _pages(g, B, capacity, P):
    """Page table of B sequences of `capacity` tokens in a shuffled pool, and the pool's size: its last page is nobody's."""
    per = -(-capacity // P)
    table = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).reshape(B, per).contiguous()
    return table, B * per + 1


def _pool(g, n_pages, Hkv, P, d, filled):
    if filled:  # K with a few strong channels, as trained models have; V plain
        k = torch.randn((n_pages, Hkv, P, d), generator=g, device="cuda", dtype=torch.bfloat16)
        k = k * (1 + 5 * (torch.rand((Hkv, 1, d), generator=g, device="cuda") < 0.04)).to(torch.bfloat16)
        k, ks = _quantise(k, 32)
        v = torch.randn((n_pages, Hkv, P, d), generator=g, device="cuda", dtype=torch.bfloat16)
        v, vs = _quantise(v, d)
    else:
        k = torch.zeros((n_pages, Hkv, P, d // 2), dtype=torch.uint8, device="cuda")
        v, ks = k.clone(), torch.zeros((n_pages, Hkv, P, d // 32), dtype=torch.uint8, device="cuda")
        vs = torch.zeros((n_pages, Hkv, P, 1), dtype=torch.uint8, device="cuda")
    w = torch.zeros((n_pages, Hkv, P), dtype=torch.float32, device="cuda")
    return dict(k=k, v=v, k_scale=ks, v_scale=vs.reshape(n_pages, Hkv, P), weights=w)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, kind = dict(case), case["kind"]
    s = dict(case=c)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    d = c["d"]
    if kind == "weights":
        B, H, Hkv, N = c["B"], c["H"], c["Hkv"], c["N"]
        s.update(q=randn(B, H, N, d), k=randn(B, Hkv, N, d), scale=1.0 / math.sqrt(d))
        s["lse"] = torch.empty((B, H, N), dtype=torch.float32, device="cuda")
        late = torch.ones((N, N), dtype=torch.bool, device="cuda").triu_(1) if c["causal"] else None
        for b in range(B):
            for h in range(H):
                x = (s["q"][b, h].float() @ s["k"][b, h // (H // Hkv)].float().T).mul_(s["scale"])
                if late is not None:
                    x.masked_fill_(late, -math.inf)
                s["lse"][b, h] = torch.logsumexp(x, -1)
        return s
    if kind == "append":
        B, S = c["B"], c["S"]
        s["n_new"] = _lengths(g, B, max(1, S // 4), S)
        s["lens"] = (s["n_new"] + _lengths(g, B, 0, c["longest"] - S)).to(torch.int32)
        s["first"] = s["lens"] - s["n_new"]
        s["table"], n = _pages(g, B, c["longest"], c["P"])
        s["pool"] = _pool(g, n, c["Hkv"], c["P"], d, False)
        s["k"], s["v"] = randn(B, c["Hkv"], S, d), randn(B, c["Hkv"], S, d)
        s["w"] = torch.rand((B, c["Hkv"], S), generator=g, device="cuda") if c["weights"] else None
        return s
    s["table"], n = _pages(g, c["B"], c["longest"], c["P"])
    s["pool"] = _pool(g, n, c["Hkv"], c["P"], d, True)
    if kind == "read":
        s["lens"] = _lengths(g, c["B"], max(1, c["longest"] // 2), c["longest"])
        s["first"] = (s["lens"] - c["T"]).clamp_(min=0)
    elif kind == "decode":
        s["lens"] = _lengths(g, c["B"], c["n_q"], c["longest"], c["ragged"])
        s["q"], s["scale"] = randn(c["B"], c["H"], c["n_q"], d), 1.0 / math.sqrt(d)
        s["weights0"] = torch.rand(s["pool"]["weights"].shape, generator=g, device="cuda")
    else:
        s["lens"] = _lengths(g, c["B"], max(1, c["longest"] // 2), c["longest"])
        # a few heavy keys, a long tail, and keys that nobody has looked at yet
        w = torch.exp(2 * torch.randn(s["pool"]["weights"].shape, generator=g, device="cuda"))
        s["pool"]["weights"] = w * (torch.rand(w.shape, generator=g, device="cuda") > 0.1)
        s["to_table"], n = _pages(g, c["B"], c["keep"], c["P"])
        s["to"] = _pool(g, n, c["Hkv"], c["P"], d, False)
    return s


# -------------------------------------------------------------- the plain form

def _quantise(x, block):
    """E2M1 codes (two a byte) and scale bytes of bf16 x [..., d], one scale per `block` channels."""
    x = x.float().unflatten(-1, (-1, block))
    amax = x.abs().amax(-1, keepdim=True)
    s = (amax / torch.full_like(amax, 6.0)).clamp(max=10240.0)  # a tensor as divisor: a rounded division, not a product
    bits = s.view(torch.int32)
    bits = (bits + 0x7FFFF + ((bits >> 20) & 1)) & ~0xFFFFF  # four significant bits, to nearest even
    small = ((s + 96.0) - 96.0)  # below 2^-14: multiples of 2^-17
    byte = torch.where(s < 2.0 ** -14, (small * 2.0 ** 17).to(torch.int32), (bits >> 20) - (112 << 3))
    s = torch.where(s < 2.0 ** -14, small, bits.view(torch.float32))
    bad = ~torch.isfinite(amax)
    y = (x / torch.where(s > 0, s, torch.ones_like(s))).abs()
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = torch.where(bad | (s == 0), torch.zeros_like(code), code | (torch.signbit(x).to(torch.uint8) << 3))
    code = code.flatten(-2)
    byte = torch.where(bad, torch.full_like(byte, 255), byte)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte.squeeze(-1).to(torch.uint8)


def _values(code, byte):
    """fp32 values of codes [..., d/2] with scale bytes [..., blocks]."""
    x = torch.stack((code & 15, code >> 4), -1).flatten(-2).to(torch.int16)
    # sign, exponent and mantissa bits at a half's places: 2^-14 of the value
    x = ((-(x & 8) << 12) | ((x & 7) << 9)).view(torch.float16).float() * 2.0 ** 14
    s = (byte.to(torch.int16) << 7).view(torch.float16).float()
    return (x.unflatten(-1, (s.shape[-1], -1)) * s.unsqueeze(-1)).flatten(-2)


def _rows(t, table, P):
    """Pages [n, Hkv, P, ...] of each sequence, as [B, Hkv, tokens, ...]."""
    return t[table.long()].transpose(1, 2).flatten(2, 3)


def _range_plain(pool, lens, table, first, T):
    """bf16 K and V at positions first .. first + T - 1, zero at and past the length."""
    at = first.long()[:, None] + torch.arange(T, device="cuda")
    P, Hkv = pool["k"].shape[2], pool["k"].shape[1]
    alive = at < lens.long()[:, None]
    at = torch.where(alive, at, torch.zeros_like(at))
    page = table.long().gather(1, at // P)[:, None, :]
    head, slot = torch.arange(Hkv, device="cuda")[None, :, None], (at % P)[:, None, :]
    alive = alive[:, None, :, None]
    k = _values(pool["k"][page, head, slot], pool["k_scale"][page, head, slot])
    v = _values(pool["v"][page, head, slot], pool["v_scale"][page, head, slot][..., None])
    return torch.where(alive, k, 0.0).bfloat16(), torch.where(alive, v, 0.0).bfloat16()


def _weights_plain(s):
    c = s["case"]
    B, H, Hkv, N, first = c["B"], c["H"], c["Hkv"], c["N"], c["first"]
    q = s["q"][:, :, first:].float().reshape(B, Hkv, (H // Hkv) * (N - first), c["d"])
    x = q @ s["k"].float().transpose(-1, -2)
    x.mul_(s["scale"])
    x.sub_(s["lse"][:, :, first:].reshape(B, Hkv, -1, 1))
    x.exp_()
    if c["causal"]:
        x = x.view(B, Hkv, H // Hkv, N - first, N)
        x.masked_fill_(torch.ones((N - first, N), dtype=torch.bool, device="cuda").triu_(first + 1), 0.0)
        return x.sum((2, 3))
    return x.sum(2)


def _append_plain(s):
    c, pool = s["case"], s["pool"]
    i = torch.arange(c["S"], device="cuda")[None, :]
    at = s["first"].long()[:, None] + i
    alive = i < s["n_new"].long()[:, None]
    page = torch.where(alive, s["table"].long().gather(1, at.clamp(max=s["table"].shape[1] * c["P"] - 1) // c["P"]),
                       torch.full_like(at, pool["k"].shape[0] - 1))  # what is not alive goes to nobody's page
    slot = torch.where(alive, at % c["P"], torch.zeros_like(at))
    page, slot, head = page[:, None, :], slot[:, None, :], torch.arange(c["Hkv"], device="cuda")[None, :, None]
    kc, ks = _quantise(s["k"], 32)
    vc, vs = _quantise(s["v"], c["d"])
    pool["k"][page, head, slot] = kc
    pool["k_scale"][page, head, slot] = ks
    pool["v"][page, head, slot] = vc
    pool["v_scale"][page, head, slot] = vs.squeeze(-1)
    pool["weights"][page, head, slot] = s["w"] if s["w"] is not None else torch.zeros((), device="cuda")
    k, v = _range_plain(pool, s["lens"], s["table"], s["first"], c["S"])
    return dict(k=k, v=v, weights=pool["weights"][:-1])


def _decode_plain(s):
    c, pool = s["case"], s["pool"]
    B, H, Hkv, n_q, d = c["B"], c["H"], c["Hkv"], c["n_q"], c["d"]
    k = _values(_rows(pool["k"], s["table"], c["P"]), _rows(pool["k_scale"], s["table"], c["P"]))
    T = k.shape[2]
    x = (s["q"].float().reshape(B, Hkv, -1, d) @ k.transpose(-1, -2)).mul_(s["scale"])
    del k
    limit = s["lens"].long()[:, None] - n_q + 1 + torch.arange(n_q, device="cuda")  # keys that query t sees
    seen = torch.arange(T, device="cuda")[None, None, :] < limit[:, :, None]  # [B, n_q, T]
    x = x.view(B, Hkv, H // Hkv, n_q, T).masked_fill_(~seen[:, None, None], -math.inf).view(B, Hkv, -1, T)
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp_()
    l = p.sum(-1, keepdim=True)
    v = _values(_rows(pool["v"], s["table"], c["P"]), _rows(pool["v_scale"], s["table"], c["P"])[..., None])
    # rows behind the length hold whatever the pages held before
    v.masked_fill_((torch.arange(T, device="cuda")[None, :] >= s["lens"].long()[:, None])[:, None, :, None], 0.0)
    o = ((p @ v) / l).view(B, H, n_q, d).bfloat16()
    lse = m + l.log()
    out = dict(o=o, lse=lse.view(B, H, n_q))
    if c["accumulate"]:
        w = pool["weights"]
        w.copy_(s["weights0"])
        add = (x - lse).exp_().sum(2).unflatten(2, (-1, c["P"])).transpose(1, 2)  # [B, pages, Hkv, P]
        w.index_add_(0, s["table"].flatten().long(), add.flatten(0, 1))
        out["weights"] = w[:-1]
    return out


def _evict_plain(s):
    c, pool, to = s["case"], s["pool"], s["to"]
    keep, P, Hkv = c["keep"], c["P"], c["Hkv"]
    w = _rows(pool["weights"], s["table"], P)
    T = w.shape[2]
    at = torch.arange(T, device="cuda")[None, None, :]
    lens = s["lens"].long()[:, None, None]
    score = torch.where(at >= lens - c["recent"], math.inf, w)
    score = torch.where(at >= lens, -math.inf, score)
    order = score.argsort(dim=-1, descending=True, stable=True)[..., :keep].sort(-1).values
    alive = order < lens
    kept = torch.where(alive, order, torch.full_like(order, -1)).to(torch.int32)
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    page = s["table"].long()[:, None, :].expand(-1, Hkv, -1).gather(2, order // P)
    i = torch.arange(keep, device="cuda")[None, None, :]
    to_page = torch.where(alive, s["to_table"].long()[:, None, :].gather(2, (i // P).expand(c["B"], 1, -1)),
                          torch.full_like(order, to["k"].shape[0] - 1))
    to_slot = torch.where(alive, i % P, torch.zeros_like(order))
    to["k"][to_page, head, to_slot] = pool["k"][page, head, order % P]
    to["k_scale"][to_page, head, to_slot] = pool["k_scale"][page, head, order % P]
    to["v"][to_page, head, to_slot] = pool["v"][page, head, order % P]
    to["v_scale"][to_page, head, to_slot] = pool["v_scale"][page, head, order % P]
    to["weights"][to_page, head, to_slot] = pool["weights"][page, head, order % P]
    now = s["lens"].clamp(max=keep)
    k, v = _range_plain(to, now, s["to_table"], torch.zeros_like(now), keep)
    return dict(kept=kept, lens=now, k=k, v=v, weights=to["weights"][:-1])


def _plain(s):
    kind = s["case"]["kind"]
    if kind == "weights":
        return _weights_plain(s)
    if kind == "append":
        return _append_plain(s)
    if kind == "read":
        return _range_plain(s["pool"], s["lens"], s["table"], s["first"], s["case"]["T"])
    if kind == "decode":
        return _decode_plain(s)
    return _evict_plain(s)


# --------------------------------------------------------- the framework's calls

def _kernels(s):
    import exact_attention_32_gb300 as fa
    c = s["case"]
    kind = c["kind"]
    if kind == "weights":
        return fa.key_weights(s["q"], s["k"], s["lse"], scale=s["scale"], causal=c["causal"], first_query=c["first"])
    cache = fa.KV4Cache(**s["pool"])
    if kind == "append":
        fa.kv4_append(cache, s["k"], s["v"], s["lens"], s["table"], n_new=s["n_new"], weights=s["w"])
        k, v = fa.kv4_read(cache, s["lens"], s["table"], c["S"], first=s["first"])
        return dict(k=k, v=v, weights=cache.weights[:-1])
    if kind == "read":
        return fa.kv4_read(cache, s["lens"], s["table"], c["T"], first=s["first"])
    if kind == "decode":
        if not c["accumulate"]:
            o, lse = fa.forward_kv4(s["q"], cache, s["lens"], s["table"], scale=s["scale"])
            return dict(o=o, lse=lse)
        cache.weights.copy_(s["weights0"])
        o, lse = fa.forward_kv4(s["q"], cache, s["lens"], s["table"], scale=s["scale"], accumulate=True)
        return dict(o=o, lse=lse, weights=cache.weights[:-1])
    to = fa.KV4Cache(**s["to"])
    kept, now = fa.kv4_evict(cache, s["lens"], s["table"], to, s["to_table"], c["keep"], recent=c["recent"])
    k, v = fa.kv4_read(to, now, s["to_table"], c["keep"])
    return dict(kept=kept, lens=now, k=k, v=v, weights=to.weights[:-1])


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------- the work

def work(case):
    c, d = case, case["d"]
    token = d + d // 32 + 1  # bytes of one token-head, K and V with their scales
    if c["kind"] == "weights":
        N, first = c["N"], c["first"]
        pairs = (first + 1 + N) * (N - first) / 2 if c["causal"] else N * (N - first)
        return dict(bytes=2 * c["B"] * (c["H"] * (N - first) + c["Hkv"] * N) * d + 4 * c["B"] * c["H"] * (N - first)
                    + 4 * c["B"] * c["Hkv"] * N, flops=2 * c["B"] * c["H"] * pairs * d)
    heads = c["B"] * c["Hkv"]
    if c["kind"] == "append":  # about 5/8 of S a sequence: a quarter of S to all of it
        n = c["Hkv"] * (c["S"] + (c["B"] - 1) * (max(1, c["S"] // 4) + c["S"]) / 2)
        return dict(bytes=n * (4 * d + token + 8) + n * (token + 4 * d) + (heads * c["S"] - n) * 4 * d, flops=n * 6 * d)
    if c["kind"] == "read":
        return dict(bytes=heads * c["T"] * (token + 4 * d), flops=heads * c["T"] * 2 * d)
    if c["kind"] == "decode":
        n = c["longest"] * c["B"] if not c["ragged"] else c["longest"] + (c["B"] - 1) * (c["n_q"] + c["longest"]) / 2
        n, rows = n * c["Hkv"], c["H"] // c["Hkv"] * c["n_q"]
        io = c["B"] * c["H"] * c["n_q"] * (4 * d + 4)
        return dict(bytes=n * (token + (8 if c["accumulate"] else 0)) + io, flops=4 * n * rows * d)
    n = c["Hkv"] * (c["longest"] + (c["B"] - 1) * 0.75 * c["longest"])
    kept = heads * min(c["keep"], c["longest"])
    return dict(bytes=4 * n + kept * (2 * (token + 4) + 4) + kept * (token + 4 * d), flops=n)


# ------------------------------------------------------- the definition in 64 bits

def _exact_values(code, byte):
    """Values of codes and scale bytes by the format's definition: sign, two exponent bits, one mantissa bit; and for
    the scale five exponent bits and three mantissa bits."""
    c = torch.empty((*code.shape[:-1], 2 * code.shape[-1]), dtype=torch.int64, device=code.device)
    c[..., 0::2], c[..., 1::2] = (code & 15).long(), (code >> 4).long()
    sign, e, m = 1.0 - 2.0 * (c >> 3).double(), ((c >> 1) & 3).double(), (c & 1).double()
    x = sign * torch.where(e == 0, 0.5 * m, torch.exp2(e - 1) * (1 + 0.5 * m))
    b = byte.long()
    e, m = (b >> 3).double(), (b & 7).double()
    s = torch.where(e == 0, m * 2.0 ** -17, torch.exp2(e - 15) * (1 + m / 8))
    return x * s.repeat_interleave(x.shape[-1] // s.shape[-1], dim=-1)


def _exact_round(x, block):
    """What 4 bits hold of x: the nearest grid values, ties to the even code, all in 64 bits."""
    blocks = x.double().reshape(*x.shape[:-1], -1, block)
    grid_s = torch.tensor([m * 2.0 ** -17 for m in range(8)] + [2.0 ** (e - 15) * (1 + m / 8) for e in range(1, 31)
                          for m in range(8)], dtype=torch.float64, device=x.device)[:0xE2 + 1]

    def nearest(y, grid):
        hi = torch.searchsorted(grid, y.contiguous()).clamp(1, len(grid) - 1)
        lo, a, b = hi - 1, y - grid[hi - 1], grid[hi] - y
        return torch.where((b < a) | ((a == b) & (hi % 2 == 0)), hi, lo)

    amax = blocks.abs().amax(-1)
    # amax against six times the scale grid: no division
    s = grid_s[nearest(amax, 6 * grid_s)].unsqueeze(-1)
    # |x| / s in 64 bits meets the middle of two grid values only where x is exactly there
    y = blocks.abs() / torch.where(s > 0, s, torch.ones_like(s))
    e = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    return (e[nearest(y, e)] * s * torch.sign(blocks)).reshape(x.shape)


def exact(case, seed):
    s, c, kind = prepare(case, seed), case, case["kind"]
    if kind == "weights":
        B, H, Hkv, N, first = c["B"], c["H"], c["Hkv"], c["N"], c["first"]
        w = torch.zeros((B, Hkv, N), dtype=torch.float64, device="cuda")
        for b in range(B):
            for h in range(H):
                q, k = s["q"][b, h, first:].double(), s["k"][b, h // (H // Hkv)].double()
                p = torch.exp(s["scale"] * (q @ k.T) - s["lse"][b, h, first:, None].double())
                w[b, h // (H // Hkv)] += (torch.tril(p, diagonal=first) if c["causal"] else p).sum(0)
        return w
    pool, table, P = s["pool"], s["table"].long(), c["P"]
    if kind == "append":
        T = c["S"]
        k, v = _exact_round(s["k"], 32), _exact_round(s["v"], c["d"])
        w = torch.zeros_like(pool["weights"], dtype=torch.float64)
        for b in range(c["B"]):
            n, f = int(s["n_new"][b]), int(s["first"][b])
            k[b, :, n:], v[b, :, n:] = 0, 0
            if s["w"] is not None:
                at = torch.arange(f, f + n, device="cuda")
                w[table[b, at // P], :, at % P] = s["w"][b, :, :n].T.double()
        return dict(k=k, v=v, weights=w[:-1])

    def sequence(p, tab, b, n):
        at = torch.arange(n, device="cuda")
        page, slot = tab[b, at // P], at % P
        pick = lambda t: t[page, :, slot].transpose(0, 1)  # noqa: E731  [Hkv, n, ...]
        return (_exact_values(pick(p["k"]), pick(p["k_scale"])), _exact_values(pick(p["v"]), pick(p["v_scale"])[..., None]),
                page, slot)

    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if kind == "read":
        out = torch.zeros((2, B, Hkv, c["T"], d), dtype=torch.float64, device="cuda")
        for b in range(B):
            n, f = int(s["lens"][b]), int(s["first"][b])
            k, v, _, _ = sequence(pool, table, b, n)
            m = min(c["T"], n - f)
            out[0, b, :, :m], out[1, b, :, :m] = k[:, f:f + m], v[:, f:f + m]
        return out[0], out[1]
    if kind == "decode":
        H, n_q = c["H"], c["n_q"]
        G = H // Hkv
        o = torch.zeros((B, H, n_q, d), dtype=torch.float64, device="cuda")
        lse = torch.zeros((B, H, n_q), dtype=torch.float64, device="cuda")
        w = s["weights0"].double()
        for b in range(B):
            n = int(s["lens"][b])
            k, v, page, slot = sequence(pool, table, b, n)
            for t in range(n_q):
                m = n - n_q + 1 + t
                x = s["scale"] * torch.einsum("hgd,hjd->hgj", s["q"][b, :, t].double().view(Hkv, G, d), k[:, :m])
                lse[b, :, t] = torch.logsumexp(x, -1).view(H)
                p = torch.softmax(x, -1)
                o[b, :, t] = torch.einsum("hgj,hjd->hgd", p, v[:, :m]).reshape(H, d)
                if c["accumulate"]:
                    w[page[:m], :, slot[:m]] += p.sum(1).T
        out = dict(o=o, lse=lse)
        if c["accumulate"]:
            out["weights"] = w[:-1]
        return out
    keep = c["keep"]
    out = torch.zeros((2, B, Hkv, keep, d), dtype=torch.float64, device="cuda")
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros_like(s["to"]["weights"], dtype=torch.float64)
    for b in range(B):
        n = int(s["lens"][b])
        k, v, page, slot = sequence(pool, table, b, n)
        old = pool["weights"][page, :, slot].T.double().cpu()
        m = min(keep, n)
        for h in range(Hkv):
            sure = list(range(max(0, n - c["recent"]), n))
            x = old[h].tolist()
            rest = sorted(range(max(0, n - c["recent"])), key=lambda j: (-x[j], j))[:m - len(sure)] if m > len(sure) else []
            at = torch.tensor(sorted(rest + sure[len(sure) - min(m, len(sure)):]), device="cuda")
            kept[b, h, :m] = at.to(torch.int32)
            out[0, b, h, :m], out[1, b, h, :m] = k[h, at], v[h, at]
            i = torch.arange(m, device="cuda")
            w[s["to_table"].long()[b, i // P], h, i % P] = old[h].to("cuda")[at]
    return dict(kept=kept, lens=s["lens"].clamp(max=keep), k=out[0], v=out[1], weights=w[:-1])
