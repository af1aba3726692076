"""Plain forms of the operators over an 8-bit cache (e4m3 bytes with a scale for each block of tokens and
head), in 64 bits, for the tests."""
from __future__ import annotations

import numpy as np


def _decode():
    x = np.arange(256)
    e, m = (x >> 3) & 15, x & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[(x & 127) == 127] = np.nan
    return np.where(x & 128, -v, v)


E4M3 = _decode()  # the value of each byte


def need(amax):
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    if amax == 0:
        return 2.0 ** -126
    m, e = np.frexp(amax)
    return max(2.0 ** (e - 9) if m <= 0.875 else 2.0 ** (e - 8), 2.0 ** -126)


def true_values(pool, scale):
    """The cache's values [pages, page_size, h, d]."""
    P, N = pool.shape[1], pool.shape[1] // scale.shape[1]
    return E4M3[pool] * np.repeat(scale.astype(np.float64), N, 1)[:, np.arange(P)][..., None]


def random_cache(rng, pages, P, N, h, d, spread=1.0):
    """(bytes, scales) of a cache filled with values of unlike size from block to block."""
    pool = rng.integers(0, 256, (pages, P, h, d)).astype(np.uint8)
    pool[(pool & 127) == 127] = 0x30
    scale = 2.0 ** np.round(spread * rng.standard_normal((pages, P // N, h)) - 6)
    return pool, scale.astype(np.float32)


def blocks_of(cu, used, table, P, N, num_pages):
    """For each block that new tokens fall into: (page, first row in the page, rows lo..hi that are new, token of row lo)."""
    out = []
    for b in range(len(used)):
        n = int(cu[b + 1] - cu[b])
        start, end = int(used[b]) - n, min(int(used[b]), table.shape[1] * P)
        at = max(start, 0) // N * N
        while n > 0 and at < end:
            lo, hi = max(start, at, 0), min(end, at + N)
            page = int(table[b, at // P])
            if 0 <= page < num_pages:
                out.append((page, at % P, lo - at, hi - at, int(cu[b]) + lo - start))
            at += N
    return out


def check_append(name, before, after, rows, slack, stored, cu, used, table):
    """Holds a pool after an append against the definition.  before, after: (bytes, scales); rows [T, h, d]: the new
    rows in 64 bits, slack their error bound ahead of the rounding (0: exact); stored [T]: which are stored."""
    (b8, bs), (a8, as_) = before, after
    P, N = b8.shape[1], b8.shape[1] // bs.shape[1]
    seen8, seens = np.zeros(b8.shape[:2], bool), np.zeros(bs.shape[:2], bool)
    for page, first, lo, hi, t in blocks_of(cu, used, table, P, N, b8.shape[0]):
        at = np.arange(t, t + hi - lo)
        keep = stored[at]
        if not keep.any():
            continue
        x = rows[at][keep]
        e = np.where(np.isfinite(x), np.broadcast_to(slack, rows.shape)[at][keep], 0)
        finite = np.where(np.isfinite(x), np.abs(x), 0)
        low, high = np.maximum(finite - e, 0).max((0, 2)), (finite + e).max((0, 2))
        old = bs[page, first // N].astype(np.float64)
        old = np.where(np.isfinite(old) & (old > 0) & (lo > 0), old, 0)
        s = as_[page, first // N].astype(np.float64)
        for h in range(x.shape[1]):
            assert s[h] in (max(old[h], need(low[h])), max(old[h], need(high[h]))), (name, page, first, h, s[h], old[h], low[h], high[h])
        seens[page, first // N] = True
        # a value is rounded once: half a step of e4m3 (2^-4 of the value, half of the subnormals' step 2^-9 scales)
        got = E4M3[a8[page, first + lo:first + hi][keep]] * s[:, None]
        want = np.where(np.isinf(x), np.sign(x) * 448 * s[:, None], x)
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(got), nan), name
        bound = np.maximum(2.0 ** -4 * np.abs(want), s[:, None] * 2.0 ** -10) * (1 + 2.0 ** -20) + 1.0625 * e
        err = np.abs(got - want)
        assert np.all((err <= bound) | nan), (name, page, first, float(np.nanmax(err - bound)))
        seen8[page, np.arange(first + lo, first + hi)[keep]] = True
        if lo:
            was, f = E4M3[b8[page, first:first + lo]], (old / s)[:, None]
            err = np.abs(E4M3[a8[page, first:first + lo]] - was * f)
            assert np.all(err <= np.where(f == 1, 0, np.maximum(2.0 ** -4 * np.abs(was * f), 2.0 ** -10) * (1 + 2.0 ** -20))), name
            seen8[page, first:first + lo] = True
    assert np.array_equal(b8[~seen8], a8[~seen8]), f"{name}: rows that the call has not to touch"
    assert np.array_equal(bs[~seens], as_[~seens], equal_nan=True), f"{name}: scales that the call has not to touch"
