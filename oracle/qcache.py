"""The 8-bit paged KV cache by definition (numpy, float64): what a page holds
after its tokens were written, whatever calls wrote them, and what a code
stands for.  Test infrastructure only."""
from __future__ import annotations

import numpy as np

E_MIN = -120


def e4m3_values() -> np.ndarray:
    """The 256 values of E4M3 (no infinities; 0x7F and 0xFF are NaN)."""
    c = np.arange(256)
    sign = np.where(c & 0x80, -1.0, 1.0)
    field, mant = (c >> 3) & 15, c & 7
    v = np.where(field == 0, mant * 2.0 ** -9, (8 + mant) * 2.0 ** (field - 10.0))
    v = sign * v
    v[(c & 0x7F) == 0x7F] = np.nan
    return v


def q4(x) -> np.ndarray:
    """x (BF16 values) rounded to 4 significant bits, ties to even; subnormals
    are 0, overflow stays at the largest such number, Inf and NaN are NaN."""
    x = np.asarray(x, np.float64)
    fin = np.isfinite(x)
    a = np.where(fin & (np.abs(x) >= 2.0 ** -126), x, 0.0)
    m, e = np.frexp(a)
    r = np.ldexp(np.round(m * 16), e - 4)
    top = 1.875 * 2.0 ** 127
    return np.where(fin, np.clip(r, -top, top), np.nan)


def page_scale(rows) -> float:
    """The scale of a (page, head) whose tokens so far are ``rows`` [n, 128]."""
    r = q4(rows)
    mag = np.abs(r[np.isfinite(r)])
    top = float(mag.max()) if mag.size else 0.0
    e = E_MIN if top == 0.0 else max(E_MIN, int(np.frexp(top)[1]) - 1 - 7)
    return float(2.0 ** e)


def page_codes(rows, scale) -> np.ndarray:
    """E4M3 bytes of ``rows`` under ``scale``."""
    v = q4(rows) / scale
    v = np.where(np.abs(v) < 2.0 ** -6, 0.0, v)  # NaN compares false and stays
    table = e4m3_values()[:127]
    nan = ~np.isfinite(v)
    mag = np.where(nan, 0.0, np.abs(v))
    code = np.searchsorted(table, mag)
    assert np.array_equal(table[code], mag), "a code is an E4M3 number"
    code = np.where(np.signbit(v) & (mag > 0), code | 0x80, code)
    return np.where(nan, 0x7F, code).astype(np.uint8)


def write_tokens(pool, scale, page_row, x, tokens_before=0):
    """Put the tokens x [n, hkv, 128] (positions 0 .. n - 1 of one sequence)
    into the pages ``page_row`` lists: pool [n_pages, hkv, ps, 128] uint8 and
    scale [n_pages, hkv] are changed in place, pages before the one that holds
    position ``tokens_before`` are left alone."""
    n, hkv, _ = x.shape
    ps = pool.shape[2]
    for lp in range(tokens_before // ps, (n + ps - 1) // ps):
        rows = x[lp * ps:(lp + 1) * ps]
        for h in range(hkv):
            s = page_scale(rows[:, h])
            scale[page_row[lp], h] = s
            pool[page_row[lp], h, :rows.shape[0]] = page_codes(rows[:, h], s)


def values(pool, scale) -> np.ndarray:
    """code * scale of whole pages, [n_pages, hkv, ps, 128] float64."""
    return e4m3_values()[pool] * np.asarray(scale, np.float64)[:, :, None, None]
