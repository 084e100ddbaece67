"""Plain 64-bit forms of the key-value cache's operators (numpy), for tests only.

The cache is int8 [pages, heads, page, dim] for keys and for values, and uint8 [pages,
heads, page // 16]: a block of 16 tokens stands for int8 * 2^(byte - 127). Rotation and
quantisation are defined step by step in float32, so those are computed in float32 and
compared bit for bit; the attention is computed in float64.
"""
import numpy as np

BLOCK = 16
F = np.float32


def power(byte):
    """2^(byte - 127) as float64."""
    return np.ldexp(1.0, np.asarray(byte, dtype=np.int64) - 127)


def block_byte(amax):
    """The smallest byte, from 0 on, under which amax rounds to 127 or less."""
    byte = 0
    while float(amax) >= 127.5 * float(power(byte)):
        byte += 1
    return byte


def rotate(x, pos, cos, sin, interleaved):
    """float32 x [heads, dim] of the token at pos; cos, sin float32 [positions, half] or None."""
    y = x.astype(F).copy()
    if cos is None:
        return y
    half = cos.shape[1]
    if 0 <= pos < cos.shape[0]:
        c, s = cos[pos], sin[pos]
    else:
        c = s = np.full(half, np.nan, F)
    left = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
    right = left + (1 if interleaved else half)
    a, b = y[:, left].copy(), y[:, right].copy()
    with np.errstate(all="ignore"):
        y[:, left] = (a * c).astype(F) - (b * s).astype(F)
        y[:, right] = (b * c).astype(F) + (a * s).astype(F)
    return y


def storable(x):
    x = np.where(np.isnan(x), F(0), x)
    return np.clip(x, -np.finfo(F).max, np.finfo(F).max).astype(F)


def rows_of(b, starts, lengths):
    """(first row, rows, tokens) of sequence b."""
    n = 1 if starts is None else int(starts[b + 1] - starts[b])
    return (b if starts is None else int(starts[b])), n, max(int(lengths[b]), 0)


def place(table, b, pos, page, pages):
    """(page number, token in it) of a position, or None."""
    if pos < 0 or pos // page >= table.shape[1]:
        return None
    p = int(table[b, pos // page])
    return (p, pos % page) if 0 <= p < pages else None


def append(kc, vc, ke, ve, k, v, table, lengths, starts, cos=None, sin=None, interleaved=False, q=None):
    """In place; returns the rotated q in float32 (rows of no sequence as they are)."""
    pages, heads, page, _ = kc.shape
    out = None if q is None else q.astype(F).copy()
    for b in range(table.shape[0]):
        row, n, length = rows_of(b, starts, lengths)
        p0 = length - n
        touched = {}
        for i in range(n):
            pos = p0 + i
            if q is not None:
                out[row + i] = rotate(q[row + i], pos, cos, sin, interleaved)
            at = place(table, b, pos, page, pages)
            if at:
                touched.setdefault(pos // BLOCK, []).append((at, row + i, pos))
        for blk, tokens in touched.items():
            pg, off = tokens[0][0][0], tokens[0][0][1] // BLOCK
            live = max(p0, 0) - blk * BLOCK              # earlier tokens in the block
            for kind, (cache, exp, x) in enumerate(((kc, ke, k), (vc, ve, v))):
                new = [storable(rotate(x[r], pos, cos, sin, interleaved) if kind == 0 else x[r].astype(F))
                       for _, r, pos in tokens]
                for h in range(heads):
                    byte = block_byte(max(np.abs(t[h]).max() for t in new))
                    if live > 0:
                        held = int(exp[pg, h, off])
                        byte = max(byte, held)
                        rows = slice(off * BLOCK, off * BLOCK + live)
                        cache[pg, h, rows] = np.rint(cache[pg, h, rows] * np.ldexp(1.0, held - byte))
                    for ((_, o), _, _), t in zip(tokens, new):
                        cache[pg, h, o] = np.clip(np.rint(t[h].astype(np.float64) / power(byte)), -127, 127)
                    exp[pg, h, off] = byte
    return out


def cached(cache, exp, table, b, h, count):
    """(values float64 [count, dim], which of the positions 0 .. count - 1 are there)."""
    pages, _, page, dim = cache.shape
    x, there = np.zeros((count, dim)), np.zeros(count, bool)
    for pos in range(count):
        at = place(table, b, pos, page, pages)
        if at:
            x[pos] = cache[at[0], h, at[1]].astype(np.float64) * power(exp[at[0], h, at[1] // BLOCK])
            there[pos] = True
    return x, there


def read(cache, exp, table, lengths, starts, rows):
    """float64 [rows, heads, dim], zeros where nothing is cached."""
    pages, heads, page, dim = cache.shape
    out = np.zeros((rows, heads, dim))
    for b in range(table.shape[0]):
        row, n, length = rows_of(b, starts, lengths)
        for i in range(n):
            at = place(table, b, length - n + i, page, pages)
            if at:
                out[row + i] = (cache[at[0], :, at[1]].astype(np.float64)
                                * power(exp[at[0], :, at[1] // BLOCK])[:, None])
    return out


def attention(q, kc, vc, ke, ve, table, lengths, starts, scale, causal, detail=False):
    """float64 [rows, q_heads, dim] of q (float64); rows of no sequence are NaN. With
    detail also, per row and head, sum_j p_j |v_j| / sum_j p_j (for tolerances), the
    largest scale * sum_d |q_d k_jd| and the number of tokens seen."""
    pages, heads, page, dim = kc.shape
    group = q.shape[1] // heads
    out = np.full(q.shape, np.nan)
    mag, top, seen = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape[0], np.int64)
    for b in range(table.shape[0]):
        row, n, length = rows_of(b, starts, lengths)
        count = min(length, table.shape[1] * page)
        for h in range(heads):
            if n == 0:
                continue
            k, there = cached(kc, ke, table, b, h, count)
            v, _ = cached(vc, ve, table, b, h, count)
            for i in range(n):
                lim = min(max(length - n + i + 1, 0), count) if causal else count
                use = there[:lim]
                kk, vv = k[:lim][use], v[:lim][use]
                seen[row + i] = len(kk)
                for g in range(group):
                    x = q[row + i, h * group + g]
                    if len(kk) == 0:
                        out[row + i, h * group + g] = 0
                        continue
                    s = scale * (kk @ x)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[row + i, h * group + g] = p @ vv
                    mag[row + i, h * group + g] = p @ np.abs(vv)
                    top[row + i, h * group + g] = abs(scale) * (np.abs(kk) @ np.abs(x)).max()
    return (out, mag, top, seen) if detail else out
