"""fp64 reference of the 4-bit KV cache operators (test infrastructure only).

Written from the format's definition with numpy on the CPU: grids of values and
nearest-neighbour search instead of bit arithmetic, dense loops instead of
tiles.  Shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# scale grid: five exponent bits, three mantissa bits, no sign; index = byte, up to 10240
SCALES = np.array([m * 2.0 ** -17 for m in range(8)]
                  + [2.0 ** (e - 15) * (1 + m / 8) for e in range(1, 31) for m in range(8)])[:0xE2 + 1]


def _nearest(y, grid):
    """Index of the grid value nearest to y >= 0, ties to the even index, saturating."""
    hi = np.clip(np.searchsorted(grid, y), 1, len(grid) - 1)
    a, b = y - grid[hi - 1], grid[hi] - y
    return np.where((b < a) | ((a == b) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x, block):
    """(packed codes uint8 [..., d/2], scale bytes uint8 [..., d/block]) of x [..., d]."""
    x = np.asarray(x, dtype=np.float64)
    xb = x.reshape(*x.shape[:-1], -1, block)
    bad = ~np.isfinite(xb).all(-1)
    safe = np.where(bad[..., None], 0.0, xb)
    byte = _nearest(np.abs(safe).max(-1), 6 * SCALES)
    s = SCALES[byte][..., None]
    code = np.where(s > 0, _nearest(np.abs(safe) / np.where(s > 0, s, 1.0), E2M1) | (np.signbit(safe) << 3), 0)
    code = np.where(bad[..., None], 0, code).reshape(x.shape)
    return ((code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8), np.where(bad, 255, byte).astype(np.uint8))


def values(codes, scale_bytes):
    """fp64 values of packed codes [..., d/2] under scale bytes [..., blocks]."""
    c = np.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=np.int64)
    c[..., 0::2], c[..., 1::2] = codes & 15, codes >> 4
    x = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.full(256, np.nan)  # bytes past the grid are no scales: 248.. read as infinities and NaNs of a half
    s[:len(SCALES)] = SCALES
    s = s[scale_bytes]
    return x * np.repeat(s, x.shape[-1] // s.shape[-1], axis=-1)


def rows(pages, table_row, n, page_size):
    """Tokens 0 .. n - 1 of one sequence: pages [n_pages, Hkv, P, ...] -> [Hkv, n, ...]."""
    j = np.arange(n)
    return np.moveaxis(pages[table_row[j // page_size], :, j % page_size], 0, 1)


def attention(q, k, v, scale, length):
    """One sequence: q [H, n_q, d], k, v [Hkv, length, d] -> O, LSE, per-key weight [Hkv, length], and
    what rounding bounds are made of: sum |q k| scale and sum |k| max |q| scale (largest over the keys a row admits),
    sum p |v|, and the softmax's sum with the largest term 1."""
    H, n_q, d = q.shape
    Hkv = k.shape[0]
    G = H // Hkv
    o, lse = np.zeros((H, n_q, d)), np.full((H, n_q), -np.inf)
    w, reach, spread = np.zeros((Hkv, length)), np.zeros((H, n_q)), np.zeros((H, n_q, d))
    top_q, total = np.zeros((H, n_q)), np.ones((H, n_q))
    for h in range(H):
        for t in range(n_q):
            m = length - n_q + 1 + t
            if m <= 0:
                continue
            kk, vv = k[h // G, :m], v[h // G, :m]
            s = scale * (kk @ q[h, t])
            top = s.max()
            e = np.exp(s - top)
            p = e / e.sum()
            o[h, t], lse[h, t] = p @ vv, top + np.log(e.sum())
            w[h // G, :m] += p
            reach[h, t], spread[h, t] = scale * (np.abs(kk) @ np.abs(q[h, t])).max(), p @ np.abs(vv)
            top_q[h, t], total[h, t] = scale * np.abs(q[h, t]).max() * np.abs(kk).sum(-1).max(), e.sum()
    return dict(o=o, lse=lse, weights=w, reach=reach, spread=spread, top_q=top_q, total=total)


def evict(weights, length, keep, recent):
    """Positions of one (sequence, key head) that stay, ascending."""
    first = max(0, length - recent)
    sure = list(range(first, length))
    room = min(keep, length) - len(sure)
    order = sorted(range(first), key=lambda j: (not np.isnan(weights[j]), -weights[j] if not np.isnan(weights[j]) else 0, j))
    return np.array(sorted(order[:room]) + sure, dtype=np.int64)


def key_weights(q, k, lse, scale, causal, first_query):
    """w [B, Hkv, N] from q [B, H, N, d], k [B, Hkv, N, d], lse [B, H, N]; and the largest sum |q k| scale of a key."""
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    w, reach = np.zeros((B, Hkv, N)), np.zeros((B, Hkv, N))
    for b in range(B):
        for h in range(H):
            g = h // (H // Hkv)
            s = scale * (q[b, h] @ k[b, g].T)
            on = np.ones((N, N), dtype=bool)
            if causal:
                on = np.tril(on)
            on[:first_query] = False
            on[lse[b, h] == -np.inf] = False
            w[b, g] += np.where(on, np.exp(np.where(on, s - np.where(on.any(-1), lse[b, h], 0)[:, None], 0)), 0).sum(0)
            reach[b, g] = np.maximum(reach[b, g], scale * (np.abs(q[b, h]) @ np.abs(k[b, g]).T).max(0))
    return w, reach
