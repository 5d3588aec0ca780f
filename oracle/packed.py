"""fp64 reference of attention over packed sequences with grouped heads (test infrastructure only).

Written from the definition with numpy on the CPU, a head and a sequence at a time; beside each result what
bounds on rounding are made of.  Shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def _admitted(n, causal):
    return np.tril(np.ones((n, n), dtype=bool)) if causal else np.ones((n, n), dtype=bool)


def forward(q, k, v, cu, scale, causal):
    """q [T, H, d], k, v [T, Hkv, d], offsets cu -> o, lse [H, T] (0 and -inf in rows of no sequence), and
    reach [H, T]  the largest scale sum |q k| over the row's keys;  spread [T, H, d]  sum p |v|."""
    T, H, d = q.shape
    G = H // k.shape[1]
    out = dict(o=np.zeros((T, H, d)), lse=np.full((H, T), -np.inf), reach=np.zeros((H, T)), spread=np.zeros((T, H, d)))
    for a, e in zip(cu[:-1], cu[1:]):
        if e == a:
            continue
        on = _admitted(e - a, causal)
        for h in range(H):
            qq, kk, vv = q[a:e, h], k[a:e, h // G], v[a:e, h // G]
            s = np.where(on, scale * (qq @ kk.T), -np.inf)
            top = s.max(-1, keepdims=True)
            lse = top + np.log(np.exp(s - top).sum(-1, keepdims=True))
            p = np.exp(s - lse)
            out["o"][a:e, h], out["lse"][h, a:e] = p @ vv, lse[:, 0]
            out["spread"][a:e, h] = p @ np.abs(vv)
            out["reach"][h, a:e] = np.where(on, scale * (np.abs(qq) @ np.abs(kk).T), 0).max(-1)
    return out


def backward(q, k, v, o, lse, dout, cu, scale, causal):
    """dq, dk, dv of sum(O dout) from the saved o and lse, and per gradient what its bounds are made of:
    x_abs   the sum of its terms' magnitudes
    x_p     the same with each P's relative error exp(e) - 1, e = 2^-23 times what the exponent's sums reach (a unit of
            d + 16 for S's sum, |LSE| for its product)
    x_ds    the sum of |error of dP - D| P times the other factor, in units of 2^-23 (d + 16) (dq and dk only)"""
    T, H, d = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    shape = dict(dq=(T, H, d), dk=(T, Hkv, d), dv=(T, Hkv, d))
    r = {x + y: np.zeros(shape[x]) for x in shape for y in ("", "_abs", "_p", "_ds")}
    for a, e in zip(cu[:-1], cu[1:]):
        if e == a:
            continue
        on = _admitted(e - a, causal)
        for h in range(H):
            g = h // G
            qq, kk, vv, go = q[a:e, h], k[a:e, g], v[a:e, g], dout[a:e, h]
            p = np.where(on, np.exp(np.where(on, scale * (qq @ kk.T), -np.inf) - lse[h, a:e, None]), 0)
            dp, row = go @ vv.T, (go * o[a:e, h]).sum(-1, keepdims=True)
            ds = p * (dp - row)
            ep = ((d + 16) * scale * (np.abs(qq) @ np.abs(kk).T) + 2 * np.abs(lse[h, a:e, None]) + 4) * 2.0 ** -23
            eds = p * (np.abs(go) @ np.abs(vv).T + (np.abs(go) * np.abs(o[a:e, h])).sum(-1, keepdims=True))
            for y, m, pp in (("", ds, p), ("_abs", np.abs(ds), p), ("_p", np.abs(ds) * ep, p * ep), ("_ds", eds, 0 * p)):
                f = (lambda x: x) if y == "" else np.abs
                r["dq" + y][a:e, h] = scale * (m @ f(kk))
                r["dk" + y][a:e, g] += scale * (m.T @ f(qq))
                r["dv" + y][a:e, g] += pp.T @ f(go)
    return r
