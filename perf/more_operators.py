"""Packed prompts, drafted trees and page moves, as they are measured: sizes, inputs, their
plain form in elementary torch operations, the framework's calls and the definition in 64 bits.

Kinds of case (a token-head is one token of one key head):
  forward   attention of packed sequences of different lengths, grouped heads
  backward  its gradients with respect to q, k and v
  tree      attention of a tree of drafted tokens of each sequence over its 4-bit cache
  keep      drafted tokens enter the cache, the accepted path stays, and is read back
  copy      pages of the cache copied (a fork's last pages, or all of them to another pool), and read back

Packed tensors are [T, heads, d]; sequence b has the rows cu[b] .. cu[b + 1] - 1.  Lengths lie
evenly on a logarithmic scale between a case's shortest and longest, in an order that the seed
gives.  The cache: pages of P tokens, [n_pages, Hkv, P, ...]; E2M1 codes two a byte (the even
channel in the low nibble), one scale byte per 32 channels of K and one per token of V; a scale
byte is the upper magnitude bits of a half (half(byte << 7)).
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a few short questions, answered together: the call's latency
        dict(name="forward_short", kind="forward", B=3, H=8, Hkv=2, d=64, shortest=17, longest=120, causal=True, fused=True),
        # the prompts of a serving step, straight from one projection's output
        dict(name="forward_prompts", kind="forward", B=16, H=32, Hkv=8, d=128, shortest=200, longest=4096, causal=True,
             fused=True),
        # documents for an encoder: every token sees all of its own, every head has its keys
        dict(name="forward_documents", kind="forward", B=48, H=16, Hkv=16, d=64, shortest=100, longest=1000, causal=False,
             fused=False),
        # long documents beside each other
        dict(name="forward_long", kind="forward", B=3, H=32, Hkv=8, d=128, shortest=5000, longest=16384, causal=True,
             fused=False),
        # a small batch of a fine-tuning step: latency
        dict(name="backward_short", kind="backward", B=4, H=6, Hkv=2, d=64, shortest=33, longest=250, causal=True,
             fused=False),
        # a training step's batch, packed
        dict(name="backward_batch", kind="backward", B=8, H=32, Hkv=8, d=128, shortest=700, longest=4096, causal=True,
             fused=True),
        # one conversation with sixteen drafts
        dict(name="tree_one", kind="tree", B=1, H=16, Hkv=4, n_q=16, d=64, P=16, longest=700),
        # a serving batch, a tree each
        dict(name="tree_batch", kind="tree", B=32, H=32, Hkv=8, n_q=12, d=128, P=64, longest=8192),
        # what one conversation keeps of its drafts
        dict(name="keep_one", kind="keep", B=1, Hkv=4, n_q=16, d=64, P=16, longest=700),
        # what a full serving batch keeps
        dict(name="keep_batch", kind="keep", B=64, Hkv=8, n_q=32, d=128, P=64, longest=8192),
        # eight continuations of each of four prompts: the page that they do not share
        dict(name="copy_fork", kind="copy", B=4, forks=8, Hkv=8, d=128, P=64, longest=2000),
        # long sequences moved to another pool
        dict(name="copy_pool", kind="copy", B=16, forks=0, Hkv=8, d=128, P=64, longest=16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["forward", "forward", "backward", "backward", "tree", "keep", "copy"])
    d, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8])
    if kind in ("forward", "backward"):
        G = rng.choice([1, 2, 3, 4, 7, 8])
        longest = _log(rng, 1, 12000 if kind == "forward" else 4096)
        shortest = _log(rng, 1, longest)
        c = dict(kind=kind, B=_log(rng, 1, 64), H=Hkv * G, Hkv=Hkv, d=d, shortest=shortest, longest=longest,
                 causal=rng.random() < 0.7, fused=rng.random() < 0.5)
        most = max((work(x)["flops"] for x in listed() if x["kind"] == kind))
        while c["B"] > 1 and (work(c)["flops"] > most or sum(_lengths(c)) > 40000):
            c["B"] = c["B"] * 2 // 3
        while c["Hkv"] > 1 and work(c)["flops"] > most:
            c["Hkv"], c["H"] = c["Hkv"] - 1, (c["Hkv"] - 1) * G
        while work(c)["flops"] > most:
            c["longest"] = c["longest"] * 2 // 3
            c["shortest"] = min(c["shortest"], c["longest"])
        return c
    P, n_q = rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 3, 5, 8, 13, 24, 32, 64])
    longest = n_q + _log(rng, 1, 16384)
    if kind == "tree":
        G = rng.choice([1, 2, 3, 4, 7, 8])
        B = max(1, min(_log(rng, 1, 64), 32 * 8192 // longest // max(1, G * n_q // 48)))
        return dict(kind=kind, B=B, H=Hkv * G, Hkv=Hkv, n_q=n_q, d=d, P=P, longest=longest)
    B = max(1, min(_log(rng, 1, 64), 16 * 16384 // longest))
    if kind == "keep":
        return dict(kind=kind, B=B, Hkv=Hkv, n_q=n_q, d=d, P=P, longest=longest)
    return dict(kind=kind, B=B, forks=rng.choice([0, 1, 2, 5, 8]), Hkv=Hkv, d=d, P=P, longest=longest)


def _lengths(c):
    """A packed case's lengths, ascending."""
    B, lo, hi = c["B"], c["shortest"], c["longest"]
    return [hi] if B == 1 else [int(round(lo * (hi / lo) ** (i / (B - 1)))) for i in range(B)]


# ----------------------------------------------------------------- the inputs

def _pool(g, n_pages, Hkv, P, d, filled):
    """A pool of pages; filled: K with a few strong channels, as trained models have, V plain."""
    if filled:
        k = torch.randn((n_pages, Hkv, P, d), generator=g, device="cuda", dtype=torch.bfloat16)
        k = k * (1 + 5 * (torch.rand((Hkv, 1, d), generator=g, device="cuda") < 0.04)).to(torch.bfloat16)
        k, ks = _quantise(k, 32)
        v = torch.randn((n_pages, Hkv, P, d), generator=g, device="cuda", dtype=torch.bfloat16)
        v, vs = _quantise(v, d)
        w = torch.rand((n_pages, Hkv, P), generator=g, device="cuda")
    else:
        k = torch.zeros((n_pages, Hkv, P, d // 2), dtype=torch.uint8, device="cuda")
        v, ks = k.clone(), torch.zeros((n_pages, Hkv, P, d // 32), dtype=torch.uint8, device="cuda")
        vs = torch.zeros((n_pages, Hkv, P, 1), dtype=torch.uint8, device="cuda")
        w = torch.zeros((n_pages, Hkv, P), dtype=torch.float32, device="cuda")
    return dict(k=k, v=v, k_scale=ks, v_scale=vs.reshape(n_pages, Hkv, P), weights=w)


def _tables(g, B, capacity, P, extra=0):
    """Page table of B sequences of `capacity` tokens in a shuffled pool, `extra` free pages, and the pool's size: its
    last page is nobody's."""
    per = -(-capacity // P)
    pages = torch.randperm(B * per + extra, generator=g, device="cuda").to(torch.int32)
    return pages[:B * per].reshape(B, per).contiguous(), pages[B * per:].contiguous(), B * per + extra + 1


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, kind, d = dict(case), case["kind"], case["d"]
    s = dict(case=c, scale=1.0 / math.sqrt(d))
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    if kind in ("forward", "backward"):
        H, Hkv = c["H"], c["Hkv"]
        lens = _lengths(c)
        lens = [lens[i] for i in torch.randperm(len(lens), generator=g, device="cuda").tolist()]
        s["cu"] = [0]
        for n in lens:
            s["cu"].append(s["cu"][-1] + n)
        T = s["cu"][-1]
        s["cu_seqlens"] = torch.tensor(s["cu"], dtype=torch.int32, device="cuda")
        if c["fused"]:  # one projection's output
            qkv = randn(T, H + 2 * Hkv, d)
            s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        else:
            s["q"], s["k"], s["v"] = randn(T, H, d), randn(T, Hkv, d), randn(T, Hkv, d)
        if kind == "backward":
            s["dout"] = randn(T, H, d)
            s["o"], s["lse"] = _forward_plain(s)
        if own:  # the lengths' plan, which all layers of a model share
            import exact_attention_32_gb300 as fa
            s["plan"] = fa.packed_plan(s["cu_seqlens"], T, causal=c["causal"])
        return s
    B, Hkv, P = c["B"], c["Hkv"], c["P"]
    if kind == "copy":
        s["lens"] = _ragged(g, B, 1, c["longest"])
        if c["forks"]:  # each sequence's last page to a page of every fork's own; the rest is shared
            n = B * c["forks"]
            s["table"], own_pages, n_pages = _tables(g, B, c["longest"], P, extra=n)
            s["lens"] = s["lens"].repeat_interleave(c["forks"])
            s["to_table"] = s["table"].repeat_interleave(c["forks"], 0).contiguous()
            s["first"] = (s["lens"] - 1) // P * P
            last = (s["first"] // P).long()[:, None]
            s["pages"] = s["to_table"].gather(1, last)[:, 0].contiguous()
            s["to_table"].scatter_(1, last, own_pages[:, None])
            s["to_pages"] = own_pages
            s["pool"] = _pool(g, n_pages, Hkv, P, d, True)
            s["to"], s["count"] = s["pool"], P
        else:  # every page, to other places of another pool
            s["table"], _, n_pages = _tables(g, B, c["longest"], P)
            s["to_table"], _, _ = _tables(g, B, c["longest"], P)
            s["pages"], s["to_pages"] = s["table"].flatten(), s["to_table"].flatten()
            s["first"], s["count"] = torch.zeros_like(s["lens"]), c["longest"]
            s["pool"], s["to"] = _pool(g, n_pages, Hkv, P, d, True), _pool(g, n_pages, Hkv, P, d, False)
        return s
    n_q = c["n_q"]
    s["table"], _, n_pages = _tables(g, B, c["longest"], P)
    s["pool"] = _pool(g, n_pages, Hkv, P, d, True)
    s["lens"] = _ragged(g, B, n_q, c["longest"])
    # a tree for each sequence: node i hangs from one of the five before it, or begins a branch of its own
    back = torch.randint(1, 6, (B, n_q), generator=g, device="cuda").tolist()
    parent = [[i - x if x <= i else -1 for i, x in enumerate(row)] for row in back]
    if kind == "tree":
        s["q"] = randn(B, c["H"], n_q, d)
        masks = []
        for row in parent:
            m = []
            for i, p in enumerate(row):
                m.append((m[p] if p >= 0 else 0) | 1 << i)
            masks.append([x - (1 << 64) if x >> 63 else x for x in m])
        s["tree"] = torch.tensor(masks, dtype=torch.int64, device="cuda")
        return s
    # the path to a leaf, cut where the drafts stop being right
    s["k"], s["v"] = randn(B, Hkv, n_q, d), randn(B, Hkv, n_q, d)
    s["w"] = torch.rand((B, Hkv, n_q), generator=g, device="cuda")
    path = torch.zeros((B, n_q), dtype=torch.int32)
    n_path = torch.randint(1, n_q + 1, (B,), generator=g, device="cuda").tolist()
    for b, row in enumerate(parent):
        nodes, i = [], n_q - 1
        while i >= 0:
            nodes.append(i)
            i = row[i]
        n_path[b] = min(n_path[b], len(nodes))
        path[b, :n_path[b]] = torch.tensor(nodes[::-1][:n_path[b]], dtype=torch.int32)
    s["path"], s["n_path"] = path.cuda(), torch.tensor(n_path, dtype=torch.int32, device="cuda")
    s["first"] = s["lens"] - n_q
    return s


def _ragged(g, B, lo, hi):
    """B lengths in [lo, hi], the first of them hi."""
    n = torch.full((B,), hi, dtype=torch.int32, device="cuda")
    if B > 1:
        n[1:] = torch.randint(lo, hi + 1, (B - 1,), generator=g, device="cuda", dtype=torch.int32)
    return n


# -------------------------------------------------------------- the plain form

def _scores_plain(s, a, n, kv, r0, r1):
    """Scaled scores [G, rows, keys] of rows r0 .. r1 - 1 of the n rows from a on, for key head kv."""
    c = s["case"]
    G = c["H"] // c["Hkv"]
    keys = r1 if c["causal"] else n
    q = s["q"][a + r0:a + r1, kv * G:(kv + 1) * G].float().transpose(0, 1)
    x = (q @ s["k"][a:a + keys, kv].float().T).mul_(s["scale"])
    if c["causal"]:
        x.masked_fill_(torch.ones((r1 - r0, keys), dtype=torch.bool, device="cuda").triu_(r0 + 1), -math.inf)
    return x


_ROWS = 4096  # of a sequence at a time: its scores fit


def _forward_plain(s):
    c = s["case"]
    H, Hkv, d, T = c["H"], c["Hkv"], c["d"], s["cu"][-1]
    G = H // Hkv
    o = torch.empty((T, H, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((H, T), dtype=torch.float32, device="cuda")
    for a, e in zip(s["cu"], s["cu"][1:]):
        for kv in range(Hkv):
            for r0 in range(0, e - a, _ROWS):
                r1 = min(e - a, r0 + _ROWS)
                x = _scores_plain(s, a, e - a, kv, r0, r1)
                m = x.amax(-1, keepdim=True)
                x.sub_(m).exp_()
                l = x.sum(-1, keepdim=True)
                y = (x @ s["v"][a:a + x.shape[-1], kv].float()).div_(l)
                o[a + r0:a + r1, kv * G:(kv + 1) * G] = y.transpose(0, 1).bfloat16()
                lse[kv * G:(kv + 1) * G, a + r0:a + r1] = (m + l.log())[..., 0]
    return o, lse


def _backward_plain(s):
    c = s["case"]
    H, Hkv, d, T = c["H"], c["Hkv"], c["d"], s["cu"][-1]
    G = H // Hkv
    dq = torch.empty((T, H, d), dtype=torch.bfloat16, device="cuda")
    dk = torch.zeros((T, Hkv, d), dtype=torch.float32, device="cuda")
    dv = torch.zeros_like(dk)
    for a, e in zip(s["cu"], s["cu"][1:]):
        for kv in range(Hkv):
            for r0 in range(0, e - a, _ROWS):
                r1, heads = min(e - a, r0 + _ROWS), slice(kv * G, (kv + 1) * G)
                p = _scores_plain(s, a, e - a, kv, r0, r1)
                keys = slice(a, a + p.shape[-1])
                p.sub_(s["lse"][heads, a + r0:a + r1, None]).exp_()
                go = s["dout"][a + r0:a + r1, heads].float().transpose(0, 1)
                dv[keys, kv] += (p.transpose(1, 2) @ go).sum(0)
                row = (go * s["o"][a + r0:a + r1, heads].float().transpose(0, 1)).sum(-1, keepdim=True)
                ds = (go @ s["v"][keys, kv].float().T).sub_(row).mul_(p).mul_(s["scale"])
                dq[a + r0:a + r1, heads] = (ds @ s["k"][keys, kv].float()).transpose(0, 1).bfloat16()
                dk[keys, kv] += (ds.transpose(1, 2) @ s["q"][a + r0:a + r1, heads].float().transpose(0, 1)).sum(0)
    return dq, dk.bfloat16(), dv.bfloat16()


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
    y = (x / torch.where(s > 0, s, torch.ones_like(s))).abs()
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = torch.where(s == 0, torch.zeros_like(code), code | (torch.signbit(x).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte.squeeze(-1).to(torch.uint8)


def _values(code, byte):
    """fp32 values of codes [..., d/2] with scale bytes [..., blocks]."""
    x = torch.stack((code & 15, code >> 4), -1).flatten(-2).to(torch.int16)
    # sign, exponent and mantissa bits at a half's places: 2^-14 of the value
    x = ((-(x & 8) << 12) | ((x & 7) << 9)).view(torch.float16).float() * 2.0 ** 14
    s = (byte.to(torch.int16) << 7).view(torch.float16).float()
    return (x.unflatten(-1, (s.shape[-1], -1)) * s.unsqueeze(-1)).flatten(-2)


def _rows(t, table):
    """Pages [n, Hkv, P, ...] of each sequence, as [B, Hkv, tokens, ...]."""
    return t[table.long()].transpose(1, 2).flatten(2, 3)


def _read_plain(pool, lens, table, first, count):
    """bf16 K and V at positions first .. first + count - 1, zero at and past the length."""
    at = first.long()[:, None] + torch.arange(count, device="cuda")
    P, Hkv = pool["k"].shape[2], pool["k"].shape[1]
    alive = at < lens.long()[:, None]
    at = torch.where(alive, at, torch.zeros_like(at))
    page = table.long().gather(1, at // P)[:, None, :]
    head, slot = torch.arange(Hkv, device="cuda")[None, :, None], (at % P)[:, None, :]
    alive = alive[:, None, :, None]
    k = _values(pool["k"][page, head, slot], pool["k_scale"][page, head, slot])
    v = _values(pool["v"][page, head, slot], pool["v_scale"][page, head, slot][..., None])
    return torch.where(alive, k, 0.0).bfloat16(), torch.where(alive, v, 0.0).bfloat16()


def _tree_plain(s):
    c, pool = s["case"], s["pool"]
    B, H, Hkv, n_q, d = c["B"], c["H"], c["Hkv"], c["n_q"], c["d"]
    k = _values(_rows(pool["k"], s["table"]), _rows(pool["k_scale"], s["table"]))
    T = k.shape[2]
    x = (s["q"].float().reshape(B, Hkv, -1, d) @ k.transpose(-1, -2)).mul_(s["scale"])
    del k
    draft = torch.arange(T, device="cuda")[None, :] - (s["lens"].long()[:, None] - n_q)  # its number, negative: context
    bit = (s["tree"][:, :, None] >> draft.clamp(0, 63)[:, None, :]) & 1
    seen = (draft[:, None, :] < 0) | ((draft[:, None, :] < n_q) & (bit != 0))  # [B, n_q, T]
    x = x.view(B, Hkv, H // Hkv, n_q, T).masked_fill_(~seen[:, None, None], -math.inf).view(B, Hkv, -1, T)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    v = _values(_rows(pool["v"], s["table"]), _rows(pool["v_scale"], s["table"])[..., None])
    o = ((x @ v) / l).view(B, H, n_q, d).bfloat16()
    return dict(o=o, lse=(m + l.log()).view(B, H, n_q))


def _keep_plain(s):
    c, pool, P = s["case"], s["pool"], s["case"]["P"]
    head = torch.arange(c["Hkv"], device="cuda")[None, :, None]

    def place(at):
        return s["table"].long().gather(1, at // P)[:, None, :], head, (at % P)[:, None, :]
    at = s["first"].long()[:, None] + torch.arange(c["n_q"], device="cuda")
    here = place(at)
    pool["k"][here], pool["k_scale"][here] = _quantise(s["k"], 32)
    pool["v"][here], scale = _quantise(s["v"], c["d"])
    pool["v_scale"][here], pool["weights"][here] = scale.squeeze(-1), s["w"]
    # what is not of the path stays where it is
    i = torch.arange(c["n_q"], device="cuda")[None, :]
    path = torch.where(i < s["n_path"].long()[:, None], s["path"].long(), i)
    there = place(s["first"].long()[:, None] + path)
    rows = {name: t[there] for name, t in pool.items()}
    for name, t in pool.items():
        t[here] = rows[name]
    lens = s["first"] + s["n_path"]
    k, v = _read_plain(pool, lens, s["table"], s["first"], c["n_q"])
    return dict(lens=lens, k=k, v=v, weights=pool["weights"][:-1])


def _copy_plain(s):
    for name, t in s["pool"].items():
        s["to"][name][s["to_pages"].long()] = t[s["pages"].long()]
    k, v = _read_plain(s["to"], s["lens"], s["to_table"], s["first"], s["count"])
    return dict(k=k, v=v, weights=s["to"]["weights"][:-1])


_PLAIN = dict(forward=_forward_plain, backward=_backward_plain, tree=_tree_plain, keep=_keep_plain, copy=_copy_plain)


# --------------------------------------------------------- the framework's calls

def _kernels(s):
    import exact_attention_32_gb300 as fa
    c, kind = s["case"], s["case"]["kind"]
    if kind == "forward":
        return fa.forward_packed(s["q"], s["k"], s["v"], s["cu_seqlens"], scale=s["scale"], causal=c["causal"], plan=s["plan"])
    if kind == "backward":
        return fa.backward_packed(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"], s["cu_seqlens"], scale=s["scale"],
                                  causal=c["causal"], plan=s["plan"])
    cache = fa.KV4Cache(**s["pool"])
    if kind == "tree":
        o, lse = fa.forward_kv4_tree(s["q"], cache, s["lens"], s["table"], s["tree"], scale=s["scale"])
        return dict(o=o, lse=lse)
    if kind == "keep":
        fa.kv4_append(cache, s["k"], s["v"], s["lens"], s["table"], weights=s["w"])
        lens = fa.kv4_keep(cache, s["lens"], s["table"], s["path"], s["n_path"])
        k, v = fa.kv4_read(cache, lens, s["table"], c["n_q"], first=s["first"])
        return dict(lens=lens, k=k, v=v, weights=cache.weights[:-1])
    to = fa.KV4Cache(**s["to"])
    fa.kv4_copy_pages(cache, s["pages"], to, s["to_pages"])
    k, v = fa.kv4_read(to, s["lens"], s["to_table"], s["count"], first=s["first"])
    return dict(k=k, v=v, weights=to.weights[:-1])


def run(state):
    return _kernels(state) if own else _PLAIN[state["case"]["kind"]](state)


# ------------------------------------------------------------------- the work

def work(case):
    c, d, kind = case, case["d"], case["kind"]
    if kind in ("forward", "backward"):
        lens = _lengths(c)
        T, H, Hkv = sum(lens), c["H"], c["Hkv"]
        pairs = sum(n * (n + 1) / 2 if c["causal"] else n * n for n in lens)
        if kind == "forward":
            return dict(bytes=T * (4 * H * d + 4 * Hkv * d + 4 * H), flops=4 * H * pairs * d)
        return dict(bytes=T * (8 * H * d + 8 * Hkv * d + 4 * H), flops=10 * H * pairs * d)
    token = d + d // 32 + 1  # bytes of one token-head, K and V with their scales
    B, Hkv, longest = c["B"], c["Hkv"], c["longest"]
    if kind == "copy":  # pages with their weights, and what is read back of them
        pages, n = ((B * c["forks"], B * c["forks"] * c["P"] / 2) if c["forks"] else
                    (B * -(-longest // c["P"]), longest * (B + 1) / 2))
        return dict(bytes=Hkv * (pages * c["P"] * 2 * (token + 4) + n * token + (B * (c["forks"] or longest // c["P"] + 1)
                                                                                 * c["P"]) * 4 * d),
                    flops=Hkv * n * 2 * d)
    n_q = c["n_q"]
    if kind == "keep":  # the append, at most half of the drafts moved, the read
        rows = B * Hkv * n_q
        return dict(bytes=rows * (4 * d + 4 + token + 4) + rows / 2 * 2 * (token + 4) + rows * (token / 2 + 4 * d),
                    flops=rows * 6 * d)
    n = Hkv * (longest + (B - 1) * (n_q + longest) / 2)
    return dict(bytes=n * token + B * c["H"] * n_q * (4 * d + 4) + 8 * B * n_q, flops=4 * n * c["H"] // Hkv * n_q * d)


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
    s = grid_s[nearest(amax, 6 * grid_s)].unsqueeze(-1)  # amax against six times the scale grid: no division
    y = blocks.abs() / torch.where(s > 0, s, torch.ones_like(s))
    e = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    return (e[nearest(y, e)] * s * torch.sign(blocks)).reshape(x.shape)


def _softmax64(x):
    """exp(x - LSE) and LSE along the last axis, in 64 bits."""
    m = x.max(-1, keepdim=True).values
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    return torch.exp(x - lse), lse[..., 0]


def _exact_packed(s, c, backward):
    H, Hkv, d, T = c["H"], c["Hkv"], c["d"], s["cu"][-1]
    o = torch.empty((T, H, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((H, T), dtype=torch.float64, device="cuda")
    dk, dv = (torch.zeros((T, Hkv, d), dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(c["B"]):
        rows = slice(s["cu"][b], s["cu"][b + 1])
        n = rows.stop - rows.start
        for h in range(H):
            q, k, v = s["q"][rows, h].double(), s["k"][rows, h * Hkv // H].double(), s["v"][rows, h * Hkv // H].double()
            x = s["scale"] * torch.einsum("id,jd->ij", q, k)
            if c["causal"]:
                i = torch.arange(n, device="cuda")
                x[i[None, :] > i[:, None]] = -math.inf
            if not backward:
                p, lse[h, rows] = _softmax64(x)
                o[rows, h] = p @ v
                continue
            # the gradients that the call defines: P from the saved LSE, D from the saved O
            p = torch.exp(x - s["lse"][h, rows].double()[:, None])
            go = s["dout"][rows, h].double()
            ds = p * (go @ v.T - (go * s["o"][rows, h].double()).sum(1)[:, None])
            o[rows, h] = s["scale"] * (ds @ k)
            dk[rows, h * Hkv // H] += s["scale"] * (ds.T @ q)
            dv[rows, h * Hkv // H] += p.T @ go
    return (o, dk, dv) if backward else (o, lse)


def exact(case, seed):
    c, kind = case, case["kind"]
    if kind in ("forward", "backward"):
        if c["H"] * sum(n * n for n in _lengths(c)) * c["d"] * (10 if kind == "backward" else 4) > 5e12:
            return None  # too long in 64 bits
        return _exact_packed(prepare(case, seed), c, kind == "backward")
    s = prepare(case, seed)
    B, Hkv, d, P, pool, table = c["B"], c["Hkv"], c["d"], c["P"], s["pool"], s["table"].long()

    def sequence(p, tab, b, n):
        at = torch.arange(n, device="cuda")
        page, slot = tab[b, at // P], at % P
        pick = lambda t: t[page, :, slot].transpose(0, 1)  # noqa: E731  [Hkv, n, ...]
        return _exact_values(pick(p["k"]), pick(p["k_scale"])), _exact_values(pick(p["v"]), pick(p["v_scale"])[..., None])

    if kind == "tree":
        H, n_q = c["H"], c["n_q"]
        o = torch.zeros((B, H, n_q, d), dtype=torch.float64, device="cuda")
        lse = torch.zeros((B, H, n_q), dtype=torch.float64, device="cuda")
        for b in range(B):
            n = int(s["lens"][b])
            k, v = sequence(pool, table, b, n)
            for t, mask in enumerate(s["tree"][b].tolist()):
                seen = torch.tensor([j for j in range(n) if j < n - n_q or (mask >> (j - n + n_q)) & 1], device="cuda")
                x = s["scale"] * torch.einsum("hgd,hjd->hgj", s["q"][b, :, t].double().view(Hkv, H // Hkv, d), k[:, seen])
                p, l = _softmax64(x)
                lse[b, :, t] = l.reshape(H)
                o[b, :, t] = torch.einsum("hgj,hjd->hgd", p, v[:, seen]).reshape(H, d)
        return dict(o=o, lse=lse)
    w = s["pool" if kind == "keep" else "to"]["weights"].double()
    if kind == "keep":
        n_q = c["n_q"]
        out = torch.zeros((2, B, Hkv, n_q, d), dtype=torch.float64, device="cuda")
        k, v = _exact_round(s["k"], 32), _exact_round(s["v"], d)
        for b in range(B):
            f, m = int(s["first"][b]), int(s["n_path"][b])
            keep = s["path"][b, :m].long()
            out[0, b, :, :m], out[1, b, :, :m] = k[b, :, keep], v[b, :, keep]
            drafts = s["w"][b].double().clone()
            drafts[:, :m] = s["w"][b][:, keep].double()
            at = torch.arange(f, f + n_q, device="cuda")
            w[table[b, at // P], :, at % P] = drafts.T
        return dict(lens=s["first"] + s["n_path"], k=out[0], v=out[1], weights=w[:-1])
    n = len(s["lens"])
    out = torch.zeros((2, n, Hkv, s["count"], d), dtype=torch.float64, device="cuda")
    source = torch.arange(B, device="cuda").repeat_interleave(max(1, c["forks"]))
    for b in range(n):
        f, m = int(s["first"][b]), int(s["lens"][b])
        k, v = sequence(pool, table, int(source[b]), m)
        out[0, b, :, :m - f], out[1, b, :, :m - f] = k[:, f:], v[:, f:]
    for a, z in zip(s["pages"].tolist(), s["to_pages"].tolist()):
        w[z] = pool["weights"][a].double()
    return dict(k=out[0], v=out[1], weights=w[:-1])
