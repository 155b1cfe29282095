"""Differential attention in FP64, one sequence at a time, from its definition.

    O_m = softmax(scale q_m k_m^T) v,  out = O_1 - lam[h] O_2

with q_m, k_m the halves of a 128-wide head, causal and bottom-right aligned.
Beside the values each function returns how far an FP32 evaluation of the same
formulas may be off: sums of absolute values times the roundings that reach
them, worst case, nothing measured.
"""
from __future__ import annotations

import numpy as np

D, M = 128, 64


def _weights(q, k, scale, m):
    """Weights [nq, nk] of one head's map m, their log sums, and the relative
    error of a weight: 64 products summed in FP32 (2^-23 a step, should the
    sum truncate), the scaling (2 roundings), the exponential (2^-22), each
    once in the weight and once in the sum."""
    nq, nk = q.shape[0], k.shape[0]
    a, b = q[:, m * M:(m + 1) * M], k[:, m * M:(m + 1) * M]
    s = scale * (a @ b.T)
    seen = np.tri(nq, nk, nk - nq, dtype=bool)
    s = np.where(seen, s, -np.inf)
    top = s.max(1)
    p = np.exp(s - top[:, None])
    lse = top + np.log(p.sum(1))
    size = scale * (np.abs(a) @ np.abs(b).T)
    err = 2 * (64 * 2.0 ** -23 * np.where(seen, size, 0).max(1) + 2.0 ** -22 * (1 + np.abs(np.where(seen, s, 0)).max(1)))
    return p / p.sum(1)[:, None], lse, err


def _fold(nk):
    """The fold of a row's block states, relative: per block, two factors by the
    hardware's exponential (2^-22 each) and a few roundings, once in the
    weighted sum and once in the sum of the weights."""
    return 2 * (-(-nk // 128) + 2) * (2 * 2.0 ** -22 + 4 * 2.0 ** -24)


def forward(q, k, v, lam, scale):
    """q [nq, Hq, 128], k, v [nk, Hkv, 128], lam [Hq] -> out, out2, lse, and the
    bounds of each."""
    q, k, v, lam = (np.asarray(x, np.float64) for x in (q, k, v, lam))
    nq, hq, nk, g = q.shape[0], q.shape[1], k.shape[0], q.shape[1] // k.shape[1]
    out, out2, lse = np.zeros((nq, hq, D)), np.zeros((nq, hq, D)), np.zeros((nq, hq, 2))
    tol, tol2, tol_lse = np.zeros_like(out), np.zeros_like(out), np.zeros_like(lse)
    for h in range(hq):
        o, t = [], []
        for m in range(2):
            p, l, e = _weights(q[:, h], k[:, h // g], scale, m)
            vv = v[:, h // g]
            # P in two BF16 pieces (2^-18), 256 products summed in FP32 (2^-15)
            rel = e + _fold(nk) + 2.0 ** -15 + 2.0 ** -18
            o.append(p @ vv)
            t.append(rel[:, None] * (p @ np.abs(vv)))
            lse[:, h, m] = l
            tol_lse[:, h, m] = e + _fold(nk) + 2.0 ** -20 + 2.0 ** -23 * np.abs(l)
        out[:, h] = o[0] - lam[h] * o[1]
        out2[:, h] = o[1]
        tol2[:, h] = t[1]
        tol[:, h] = t[0] + abs(lam[h]) * t[1] + 2.0 ** -23 * np.abs(out[:, h])
    return out, out2, lse, tol, tol2, tol_lse


def backward(q, k, v, lam, dout, scale):
    """Whole sequences (nq = nk): dq, dk, dv, dlam, and the bounds of each."""
    q, k, v, lam, dout = (np.asarray(x, np.float64) for x in (q, k, v, lam, dout))
    n, hq, g = q.shape[0], q.shape[1], q.shape[1] // k.shape[1]
    dq, dk, dv, dlam = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros(hq)
    tq, tk, tv, tl = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros(hq)
    out, out2, _, tol, tol2, _ = forward(q, k, v, lam, scale)
    total = 2 * (n + 127) // 128 * 128 * 2.0 ** -23  # FP32 sums over a row's or a column's products, hi and lo
    for h in range(hq):
        kv, do = h // g, dout[:, h]
        vv = v[:, kv]
        dp, dp_abs = do @ vv.T, np.abs(do) @ np.abs(vv).T
        for m, c in ((0, 1.0), (1, -lam[h])):
            cols = slice(m * M, (m + 1) * M)
            p, l, e = _weights(q[:, h], k[:, kv], scale, m)
            # a weight from the saved log sum, which has its own error
            rel = (2 * e + _fold(n) + 2.0 ** -21 * (1 + np.abs(l)))[:, None]
            delta = (p * dp).sum(1, keepdims=True)
            o = p @ vv
            # Delta from the saved outputs: their error, and sums of 128 products
            t_o = tol2[:, h] if m else tol[:, h] + abs(lam[h]) * tol2[:, h]
            o_abs = np.abs(o) if m else np.abs(out[:, h]) + abs(lam[h]) * np.abs(out2[:, h])
            t_delta = (np.abs(do) * (t_o + 2.0 ** -16 * o_abs)).sum(1, keepdims=True)
            pc = c * p
            ds = pc * (dp - delta)
            t_ds = np.abs(pc) * ((rel + 2.0 ** -18 + 2.0 ** -22) * np.abs(dp - delta) + 2.0 ** -16 * dp_abs + t_delta)
            dv[:, kv] += pc.T @ do
            tv[:, kv] += np.abs(pc * (rel + 2.0 ** -18 + total * g)).T @ np.abs(do)
            dq[:, h, cols] = scale * (ds @ k[:, kv, cols])
            tq[:, h, cols] = scale * ((t_ds + total * np.abs(ds)) @ np.abs(k[:, kv, cols]))
            dk[:, kv, cols] += scale * (ds.T @ q[:, h, cols])
            tk[:, kv, cols] += scale * ((t_ds + total * g * np.abs(ds)).T @ np.abs(q[:, h, cols]))
            if m:
                dlam[h] = -delta.sum()
                tl[h] = t_delta.sum() + n * 2.0 ** -24 * np.abs(delta).sum()
    return dq, dk, dv, dlam, tq, tk, tv, tl
