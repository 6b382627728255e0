"""Float64 NumPy definitions of the decoding operators (test infrastructure
only): the block layout of the 8-bit paged key/value cache, appending to it
with rotation by position, and attention over it. Nothing here shares code
with the library."""
import numpy as np


def k_place(t, d, D):
    """Byte of token t, dimension d in a block of keys."""
    return (t // 16) * 16 * D + (d // 16) * 256 + (t % 16) * 16 + d % 16


def v_place(t, d, D):
    """Byte of token t, dimension d in a block of values."""
    return (t // 4) * 4 * D + 4 * d + t % 4


def block_codes(block, which, page, D):
    """Signed codes [page, D] of one block's bytes."""
    t, d = np.meshgrid(np.arange(page), np.arange(D), indexing="ij")
    at = k_place(t, d, D) if which == "k" else v_place(t, d, D)
    return np.asarray(block).reshape(-1)[at].astype(np.int64) - 128


def block_bytes(codes, which):
    """Bytes [page * D] of signed codes [page, D]."""
    page, D = codes.shape
    t, d = np.meshgrid(np.arange(page), np.arange(D), indexing="ij")
    out = np.empty(page * D, dtype=np.uint8)
    out[k_place(t, d, D) if which == "k" else v_place(t, d, D)] = (codes + 128).astype(np.uint8)
    return out


def rotate(x, pos, cos, sin, interleaved):
    """Rows x [n, heads, D] at positions pos [n], float64."""
    y = np.array(x, dtype=np.float64)
    half = cos.shape[1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = (m[pos, i].astype(np.float64)[:, None] for m in (cos, sin))
        y[:, :, a], y[:, :, b] = x[:, :, a] * c - x[:, :, b] * s, x[:, :, a] * s + x[:, :, b] * c
    return y


def append_block(codes, scale, first, rows):
    """One block [page, D] with `scale`: rows go to tokens first, first + 1, ...
    Returns (codes, scale)."""
    page, D = codes.shape
    rows = np.where(np.isfinite(rows), rows, 0.0)
    old = float(scale) if first else 0.0
    new = max(old, np.abs(rows).max() / 127.0)
    if new < 2.0 ** -100:
        new = 0.0
    codes = codes.copy()
    if first and new != old:
        codes[:first] = np.rint(codes[:first] * (old / new if new else 0.0)).astype(np.int64)
    codes[first:first + len(rows)] = np.clip(np.rint(rows / new), -127, 127) if new else 0
    return codes, new


def cache_rows(cache, scales, table_row, which, lo, hi):
    """Values [hi - lo, heads, D] (float64) of tokens lo .. hi - 1 of one sequence;
    NaN where there is no page."""
    pages, H, page, D = cache.shape
    out = np.full((hi - lo, H, D), np.nan)
    for t in range(lo, hi):
        slot = t // page
        if slot >= len(table_row) or not 0 <= table_row[slot] < pages:
            continue
        p = table_row[slot]
        d = np.arange(D)
        at = k_place(t % page, d, D) if which == "k" else v_place(t % page, d, D)
        for h in range(H):
            out[t - lo, h] = (cache[p, h].reshape(-1)[at].astype(np.float64) - 128) * np.float64(scales[p, h])
    return out


def attention(q, k, v, vs, first_pos, scale, causal, window):
    """q [n, Hq, D] at positions first_pos .. over k, v [L, H, D] (float64; a token
    whose page does not exist is NaN in k) with value scales vs [L, H]. Returns out,
    lse, sum p |v| / sum p, and tokens * 127 * max(p vs) / sum p."""
    n, Hq, D = q.shape
    L, H, _ = k.shape
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    mag, peak = np.zeros((n, Hq, D)), np.zeros((n, Hq, 1))
    there = ~np.isnan(k).any(axis=(1, 2)) if L else np.zeros(0, bool)
    j = np.arange(L)
    for i in range(n):
        p = first_pos + i
        seen = there & (j < L)
        if causal:
            seen &= j <= p
        if window:
            seen &= j > p - window
        if not seen.any():
            continue
        for h in range(Hq):
            kk, vv = k[seen, h // (Hq // H)], v[seen, h // (Hq // H)]
            s = kk @ q[i, h] * scale
            m = s.max()
            e = np.exp(s - m)
            out[i, h] = e @ vv / e.sum()
            lse[i, h] = m + np.log(e.sum())
            mag[i, h] = e @ np.abs(vv) / e.sum()
            peak[i, h] = 127 * seen.sum() * (e * vs[seen, h // (Hq // H)]).max() / e.sum()
    return out, lse, mag, peak
