"""fp64 restatement of the 8-bit serving operators: block scales, e4m3 rounding, the norm, the
product, the cache store and the attention over it. NumPy only; test infrastructure.

An 8-bit value is kept here as the pair (e, s): e the e4m3 element as a float64 (NaN where the
element was not finite), s the block's scale 2^k; it stands for e * s.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 128


def scale_of(amax: float) -> float:
    """Smallest 2^k, k >= -126, with amax <= 448 2^k."""
    if amax == 0:
        return 2.0 ** -126
    k = max(-126, math.ceil(math.log2(amax / 448)) - 1)
    while amax > 448 * 2.0 ** k:
        k += 1
    return 2.0 ** k


def e4m3(v):
    """Nearest e4m3 value (ties to even); non-finite to NaN. |v| <= 448 + half a step."""
    v = np.asarray(v, dtype=np.float64)
    out = np.full(v.shape, np.nan)
    ok = np.isfinite(v)
    m, e = np.frexp(v[ok])                      # |v| = m 2^e, m in [0.5, 1)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))  # 3 mantissa bits; subnormals at 2^-9
    out[ok] = np.rint(v[ok] / step) * step
    return out


def quantize(x, bounds):
    """(elements, scales) of the blocks x[..., lo:hi] of the last axis for consecutive bounds."""
    x = np.asarray(x, dtype=np.float64)
    q = np.empty_like(x)
    s = np.empty(x.shape[:-1] + (len(bounds) - 1,))
    for i, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        part = x[..., lo:hi]
        amax = np.max(np.where(np.isfinite(part), np.abs(part), 0.0), axis=-1)
        f = np.vectorize(scale_of, otypes=[float])(amax)
        s[..., i] = f
        q[..., lo:hi] = e4m3(part / f[..., None])
    return q, s


def edges(n):
    return list(range(0, n, BLOCK)) + [n]


def add_rms_norm(x, delta, gain, eps, round_h):
    """(h, elements, scales). round_h rounds the sum to the rows' type."""
    h = np.asarray(x, np.float64)
    if delta is not None:
        h = round_h(h + np.asarray(delta, np.float64))
    y = h
    if gain is not None:
        with np.errstate(all="ignore"):
            y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    q, s = quantize(y, edges(h.shape[1]))
    return h, q, s


def quantize_weight(w):
    w = np.asarray(w, np.float64)
    N, K = w.shape
    q = np.empty_like(w)
    s = np.empty((-(-N // BLOCK), -(-K // BLOCK)))
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            part = w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            s[i, j] = scale_of(np.max(np.where(np.isfinite(part), np.abs(part), 0.0)))
            q[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] = e4m3(part / s[i, j])
    return q, s


def linear(xq, xs, wq, ws, resid=None):
    K, N = xq.shape[1], wq.shape[0]
    x = xq * np.repeat(xs, BLOCK, 1)[:, :K]
    w = wq * np.repeat(np.repeat(ws, BLOCK, 0)[:N], BLOCK, 1)[:, :K]
    y = x @ w.T
    return y if resid is None else y + np.asarray(resid, np.float64)


def store(cache, scale, rows, length):
    """Appends rows [n, heads, 128] behind `length` rows of one slot, in place:
    cache [cap, heads, 128] elements, scale [blocks, heads]."""
    rows = np.asarray(rows, np.float64)
    n, heads, _ = rows.shape
    if n == 0:
        return
    for blk in range(length // BLOCK, (length + n - 1) // BLOCK + 1):
        lo, hi = max(length, blk * BLOCK), min(length + n, (blk + 1) * BLOCK)
        for g in range(heads):
            part = rows[lo - length:hi - length, g]
            f = scale_of(np.max(np.where(np.isfinite(part), np.abs(part), 0.0)))
            if blk * BLOCK < length:
                f = max(f, scale[blk, g])
                if f > scale[blk, g]:
                    old = cache[blk * BLOCK:length, g]
                    cache[blk * BLOCK:length, g] = e4m3(old * (scale[blk, g] / f))
            scale[blk, g] = f
            cache[lo:hi, g] = e4m3(part / f)


def attention(q, kc, ks, vc, vs, length, group):
    """[heads * group, 128]: q rows over `length` rows of one slot (elements and scales as in
    store); zeros when length is 0."""
    heads = kc.shape[1]
    out = np.zeros((heads * group, 128))
    if length == 0:
        return out
    nb = -(-length // BLOCK)
    for g in range(heads):
        k = kc[:length, g] * np.repeat(ks[:nb, g], BLOCK)[:length, None]
        v = vc[:length, g] * np.repeat(vs[:nb, g], BLOCK)[:length, None]
        s = q[g * group:(g + 1) * group] @ k.T / math.sqrt(128)
        p = np.exp(s - s.max(1, keepdims=True))
        out[g * group:(g + 1) * group] = (p / p.sum(1, keepdims=True)) @ v
    return out
