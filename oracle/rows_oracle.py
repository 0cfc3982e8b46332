"""fp64 oracle of the row calls: norms, rotary positions and the compressor for the
newest tokens of a sequence, with bounds on what fp32 arithmetic may be off.  Plain
numpy; shares no code with the CUDA path.

Bounds count roundings in units u = 2^-24.  A sum of n terms on the GPU has at most
D = 64 additions one after another (32 in a thread, the rest across threads), so it is
off by D u times the sum of the terms' magnitudes.  A result rounded to a type of step
eps is off by eps / 2 of itself.
"""
from __future__ import annotations

import math

import numpy as np

U = 2.0 ** -24
D = 64
RMS, LAYER = 1, 2
STEP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}      # half a step of each output type


def freqs(dim, base=10000.0, scaling="plain", factor=1.0, original_len=0.0, beta_fast=32.0, beta_slow=1.0):
    f = np.array([base ** (-2.0 * i / dim) for i in range(dim // 2)])
    if scaling == "linear":
        return f / factor
    if scaling == "by_parts":
        at = lambda n: dim * math.log(original_len / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
        lo = min(max(math.floor(at(beta_fast)), 0), dim - 1)
        hi = min(max(math.ceil(at(beta_slow)), 0), dim - 1)
        g = np.clip((np.arange(dim // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        return f * (1 - g) + f / factor * g
    return f


def pairs(dim, first, half):
    """First and second channels of the pairs."""
    i = np.arange(dim // 2)
    return (first + i, first + dim // 2 + i) if half else (first + 2 * i, first + 2 * i + 1)


def turn(x, pos, f, first, half, scale, back=False):
    """(rows [..., d] turned by positions pos [...], bound of the fp32 error)."""
    u, v = pairs(2 * len(f), first, half)
    a = np.asarray(pos, np.float64)[..., None] * f * (-1 if back else 1)
    c, s = np.cos(a), np.sin(a)
    y, err = x.copy(), np.zeros_like(x)
    y[..., u] = scale * (x[..., u] * c - x[..., v] * s)
    y[..., v] = scale * (x[..., u] * s + x[..., v] * c)
    # sine and cosine 2 u, times scale, two products and a sum; the angle's own rounding on both sides
    size = abs(scale) * (np.abs(x[..., u]) + np.abs(x[..., v]))
    err[..., u] = err[..., v] = size * (6 * U + np.abs(a) * 2.0 ** -51)
    return y, err


def spread(e, f, first, half, scale):
    """A bound of rows' errors after turning them."""
    u, v = pairs(2 * len(f), first, half)
    out = e.copy()
    out[..., u] = out[..., v] = abs(scale) * (e[..., u] + e[..., v])
    return out


def _stats(x, kind, eps):
    m = x.mean(-1, keepdims=True) if kind == LAYER else np.zeros(x.shape[:-1] + (1,))
    r = 1 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    xh = (x - m) * r
    e_m = D * U * np.abs(x).mean(-1, keepdims=True) if kind == LAYER else 0 * m
    e_r = (D / 2 + 8) * U + 0.5 * (e_m * r) ** 2          # of r, relative
    return xh, r, e_m * r + np.abs(xh) * (e_r + 2 * U), e_r


def norm(x, kind, weight, bias, eps):
    """(norm of rows [..., n], bound of the fp32 error)."""
    xh, _, e, _ = _stats(x, kind, eps)
    w = np.ones(x.shape[-1]) if weight is None else weight
    b = np.zeros(x.shape[-1]) if bias is None else bias
    y = xh * w + b
    return y, e * np.abs(w) + 2 * U * (np.abs(xh * w) + np.abs(y))


def norm_bwd(x, dy, e_dy, kind, weight, eps):
    """(dx, dweight, dbias) of rows [rows, n] with gradients dy known up to e_dy, and the bounds of their errors."""
    xh, r, ex, e_r = _stats(x, kind, eps)
    w = np.ones(x.shape[-1]) if weight is None else weight
    g, eg = dy * w, e_dy * np.abs(w) + U * np.abs(dy * w)
    mean = lambda a: a.mean(-1, keepdims=True)  # noqa: E731
    mg, mgx = mean(g) * (kind == LAYER), mean(g * xh)
    e_mg = (mean(eg) + D * U * mean(np.abs(g))) * (kind == LAYER)
    e_mgx = mean(eg * np.abs(xh) + np.abs(g) * ex) + (D + 1) * U * mean(np.abs(g * xh))
    dx = r * (g - mg - xh * mgx)
    size = r * (np.abs(g) + np.abs(mg) + np.abs(xh * mgx))
    e_dx = r * (eg + e_mg + ex * np.abs(mgx) + np.abs(xh) * e_mgx) + np.abs(dx) * e_r + 4 * U * size
    rows = x.shape[0] + 16                                # additions one after another
    dw, db = (dy * xh).sum(0), dy.sum(0)
    e_dw = (e_dy * np.abs(xh) + np.abs(dy) * ex).sum(0) + rows * U * np.abs(dy * xh).sum(0)
    e_db = e_dy.sum(0) + rows * U * np.abs(dy).sum(0)
    return (dx, dw, db), (e_dx, e_dw, e_db)


def round_bf16(x):
    """fp64 values rounded to the nearest bf16, ties to even."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


def compress(kv, score, ratio, coff, kind, weight, bias, eps, f, first, half, scale, dtype):
    """Every complete block of one sequence kv [n, d], score [n, d or 1]: (rows [blocks, d], bounds of their errors).

    A pooled value next to a rounding border of bf16 may be cast either way; the bound
    then has that step, and what it does to the norm."""
    n, d = kv.shape
    out, bound = np.zeros((n // ratio, d)), np.zeros((n // ratio, d))
    for j in range(n // ratio):
        t = slice(max(0, (j + 1 - coff) * ratio), (j + 1) * ratio)
        z = np.broadcast_to(score[t], kv[t].shape)
        w = np.exp(z - z.max(0))
        w = w / w.sum(0)
        x = (w * kv[t]).sum(0)
        # A weight: its exponent is the distance to the maximum times log2 e, three roundings (of the difference, the
        # constant and the product), in the numerator and in the sum that divides it; a common offset of the scores has
        # no part in it.  8 more roundings and 16 of rescaling; the sums.
        far = w * np.where(w > 0, z.max(0) - z, 0.0)
        size = (w * np.abs(kv[t])).sum(0)
        off = (24 + 2 * D) * U * size + 3 * U * ((far * np.abs(kv[t])).sum(0) + far.sum(0) * size)
        e = off + STEP["fp32"] * np.abs(x)
        if dtype == "bf16":
            e = np.maximum(np.abs(round_bf16(x + off) - round_bf16(x)), np.abs(round_bf16(x - off) - round_bf16(x)))
            x = round_bf16(x)
        if kind:
            y, ey = norm(x, kind, weight, bias, eps)
            xh, r, _, _ = _stats(x, kind, eps)
            m = np.ones(d) if weight is None else np.abs(weight)
            mean = np.abs(e).mean() * (kind == LAYER)
            ey = ey + m * (r * (e + mean) + np.abs(xh) * (np.abs(xh) * r * (e + mean)).mean()) * (1 + 2 * (r * e).max())
        else:
            y, ey = x, e
        if f is not None:
            y, et = turn(y, (j + 1) * ratio - 1, f, first, half, scale)
            ey = spread(ey, f, first, half, scale) + et
        out[j], bound[j] = y, ey
    return out, bound
