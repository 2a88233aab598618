"""Plain form of the 4-bit key/value cache: the position rotation in fp32, what
a token's keys or values are stored as, what a cache's bytes stand for, and
attention over it in float64.

[SNIP, Fig. 4]: Q, K, V and O of a Llama-like block; between them lies the
attention that reads this cache.
"""
from __future__ import annotations

import numpy as np

from . import formats as F
from .quantize import FP4_VARIANT


def rotate(x, cos, sin, interleaved):
    """x fp32 [tokens, heads, dim]; cos, sin fp32 [tokens, rot / 2]: each
    product and sum rounded to fp32."""
    x = np.array(x, np.float32)
    half = cos.shape[1]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cos[:, None, :].astype(np.float32), sin[:, None, :].astype(np.float32)
    xa, xb = x[..., a].copy(), x[..., b].copy()
    x[..., a] = xa * c - xb * s
    x[..., b] = xb * c + xa * s
    return x


def token_major(a, keys):
    """A cache buffer's bytes [pages, heads, tokens, bytes of a token]: keys
    [pages, heads, groups, pieces, tokens, bytes], values with 4 tokens a group."""
    a = np.asarray(a)
    if a.ndim == 5:                                  # scales of values: one byte a piece
        a = a[..., None]
    pages, heads, groups, pieces, tokens, size = a.shape
    assert tokens == (16 if keys else 4)
    return a.transpose(0, 1, 2, 4, 3, 5).reshape(pages, heads, groups * tokens, pieces * size)


def values(fmt, codes, scales, texp):
    """float64 values [..., dim] of token-major codes [..., dim / 2] and scales."""
    block, kind = FP4_VARIANT[fmt]
    v = F.e2m1_decode(F.unpack_nibbles(codes.reshape(-1, codes.shape[-1]))).astype(np.float64)
    s = (F.e4m3_decode if kind == "e4m3" else F.e8m0_decode)(scales.reshape(-1, scales.shape[-1])).astype(np.float64)
    v = v * np.repeat(s, block, axis=1)
    return np.ldexp(v, texp if kind == "e4m3" else 0).reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def attention(q, k, v, pos, mapped, scale, window):
    """q [rows, heads, dim] of one kv head's query heads, k and v [tokens, dim],
    pos [rows], mapped [tokens]. Returns out and lse (-inf and 0 for a row without
    keys) and, for bounds on rounding, sum p |v|, the largest sum |q| |k| * scale
    of a key that a row sees, and the number of keys."""
    x = np.matmul(q, k.T) * scale
    size = np.matmul(np.abs(q), np.abs(k).T) * scale
    t = np.arange(k.shape[0])
    seen = (t[None] <= pos[:, None]) & mapped[None]
    if window:
        seen &= t[None] > pos[:, None] - window
    seen = np.broadcast_to(seen[:, None], x.shape)
    x = np.where(seen, x, -np.inf)  # [rows, heads, tokens]
    some = seen.any(axis=2)
    m = np.where(some, x.max(axis=2, initial=-np.inf), 0.0)
    p = np.where(seen, np.exp(x - m[..., None]), 0.0)
    total = p.sum(axis=2)
    with np.errstate(divide="ignore"):
        lse = np.where(some, m + np.log(total), -np.inf)
    p = p / np.where(some, total, 1.0)[..., None]
    v = np.where(mapped[:, None], v, 0.0)
    return (np.matmul(p, v), lse, np.matmul(p, np.abs(v)),
            np.where(seen, size, 0.0).max(axis=2, initial=0.0), seen.sum(axis=2))
