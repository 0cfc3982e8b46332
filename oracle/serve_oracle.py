"""fp64 oracle of the serving calls: the quantised paged cache, and the indexer
and attention of single tokens over it.  Plain numpy, one row at a time; shares
no code with the CUDA path.

The cache format: a group of 32 channels is codes times a power of two; bits 4:
e2m1, bits 8: e4m3.  The power of two is the smallest that holds the group's
largest magnitude (at least 2^-110, at most 2^125 or 2^119); codes round to
nearest, ties to even.
"""
from __future__ import annotations

import numpy as np

GROUP = 32
MIN_EXP = -110
MAX_EXP = {4: 125, 8: 119}


def code_grid(bits):
    """Non-negative values of the codes 0, 1, 2, ... (the sign is the top bit)."""
    if bits == 4:
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
    vals = []
    for c in range(127):                       # 127 is NaN
        e, m = c >> 3, c & 7
        vals.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(vals, dtype=np.float64)


def quantize_rows(x, bits):
    """x [..., d] -> (codes [..., d] uint8, exponents [..., d/32] int)."""
    x = np.asarray(x, dtype=np.float64)
    grid = code_grid(bits)
    codes = np.zeros(x.shape, dtype=np.uint8)
    exps = np.zeros(x.shape[:-1] + (x.shape[-1] // GROUP,), dtype=np.int64)
    for at in np.ndindex(*exps.shape):
        g = x[at[:-1]][at[-1] * GROUP:(at[-1] + 1) * GROUP]
        amax = np.abs(g).max()
        e = MIN_EXP
        while np.ldexp(grid[-1], int(e)) < amax and e < MAX_EXP[bits]:
            e += 1
        exps[at] = e
        for i, v in enumerate(g):
            a = np.ldexp(abs(v), -int(e))      # exact in fp64
            j = int(np.searchsorted(grid, a))
            if j == len(grid):
                j -= 1
            if j > 0:
                below, above = a - grid[j - 1], grid[j] - a
                if below < above or (below == above and (j - 1) % 2 == 0):
                    j -= 1
            neg = np.signbit(v)
            codes[at[:-1]][at[-1] * GROUP + i] = j | ((8 if bits == 4 else 128) if neg else 0)
    return codes, exps


def code_values(codes, exps, bits):
    """What codes and exponents stand for, fp64."""
    grid = code_grid(bits)
    top = 8 if bits == 4 else 128
    mag = grid[np.minimum(codes & (top - 1), len(grid) - 1)]
    v = np.where(codes & top, -mag, mag)
    return v * np.repeat(np.ldexp(1.0, exps), GROUP, axis=-1)


def held_rows(x, bits):
    """The rows the cache returns for x."""
    c, e = quantize_rows(x, bits)
    return code_values(c, e, bits)


def row_bytes(codes, exps, bits):
    """(code bytes [..., d*bits/8], scale bytes [..., d/32]) as the cache stores them."""
    if bits == 4:
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return codes.astype(np.uint8), (exps + 127).astype(np.uint8)


def place(pages, page_size, pos):
    """(page id, row in the page) of position pos of a sequence with the given page ids."""
    slot = pos % (len(pages) * page_size)
    return int(pages[slot // page_size]), slot % page_size


def write(cache, x, table, pos0, counts, page_size, bits):
    """The cache bytes [n_pages, page bytes] after writing x [b, s, d]."""
    out = np.array(cache, dtype=np.uint8)
    d = x.shape[-1]
    cb, sb = d * bits // 8, d // GROUP
    for s in range(x.shape[0]):
        for i in range(counts[s]):
            page, row = place(table[s], page_size, int(pos0[s]) + i)
            code, scale = row_bytes(*quantize_rows(x[s, i], bits), bits)
            out[page, row * cb:(row + 1) * cb] = code
            at = page_size * cb + row * sb
            out[page, at:at + sb] = scale
    return out


def read_row(cache, pages, page_size, bits, d, pos):
    """The values of the row at position pos, from the cache's bytes."""
    page, row = place(pages, page_size, pos)
    cb, sb = d * bits // 8, d // GROUP
    code = cache[page, row * cb:(row + 1) * cb]
    at = page_size * cb + row * sb
    exps = cache[page, at:at + sb].astype(np.int64) - 127
    if bits == 4:
        code = np.stack([code & 15, code >> 4], -1).reshape(d)
    return code_values(code, exps, bits)


def index_row(q, w, keys, t, ratio, topk):
    """The top-k blocks of one query: q [H, d], w [H], keys [n, d] (n >= vis)."""
    out = np.full(topk, -1, dtype=np.int64)
    vis = (t + 1) // ratio if t >= 0 else 0
    if vis == 0:
        return out
    dots = np.asarray(q, np.float64) @ np.asarray(keys[:vis], np.float64).T
    score = (np.maximum(dots, 0.0) * np.asarray(w, np.float64)[:, None]).sum(0)
    best = np.sort(np.argsort(-score, kind="stable")[:topk])
    out[:len(best)] = best
    return out


def attend_row(q, raw, cmp, idx, sink, scale, t, ratio, window):
    """One query: q [H, d], raw(pos) and cmp(j) return rows, idx a list of
    blocks or None (every visible one).  Returns o [H, d], lse [H] and the
    bound sum_i p_i |v_i| [H, d] of what a relative error of p moves."""
    H, d = q.shape
    rows = []
    if t >= 0:
        vis = (t + 1) // ratio
        rows = [raw(p) for p in range(max(0, t - window + 1), t + 1)]
        js = range(vis) if idx is None else [int(j) for j in idx if 0 <= j < vis]
        rows += [cmp(j) for j in js]
    sink = np.full(H, -np.inf) if sink is None else np.asarray(sink, np.float64)
    if not rows:
        return np.zeros((H, d)), sink, np.zeros((H, d))
    kv = np.stack(rows)
    z = np.concatenate([np.asarray(q, np.float64) @ kv.T * scale, sink[:, None]], 1)
    top = z.max(1, keepdims=True)
    e = np.exp(z - top)
    total = e.sum(1, keepdims=True)
    p = (e / total)[:, :-1]
    return p @ kv, (top + np.log(total))[:, 0], p @ np.abs(kv)
