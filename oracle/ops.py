"""Plain float64 forms of the operators around the quantized linear layers:
RMS norm with the residual's addition, SwiGLU, the product of a few tokens
with block-scaled weights. Inputs are numpy arrays holding the bf16 / fp32
values; nothing is rounded on the way.

[SNIP, Fig. 4]: the linear layers of a Llama-like block, whose inputs these
operators make and whose outputs they take.
"""
from __future__ import annotations

import numpy as np

from . import formats as F
from .quantize import FP4_VARIANT, FP8


def rmsnorm_fwd(x, gamma, eps, res=None):
    """h, r [rows], y."""
    h = np.asarray(x, np.float64)
    if res is not None:
        h = h + np.asarray(res, np.float64)
    r = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h, r, h * r[:, None] * np.asarray(gamma, np.float64)


def rmsnorm_bwd(dy, h, gamma, r, dres=None):
    """dx, dgamma, and the magnitudes that their rounding errors scale with:
    of each dx element's terms, and the sum of |terms| of each dgamma."""
    dy, h, gamma, r = (np.asarray(a, np.float64) for a in (dy, h, gamma, r))
    xh = h * r[:, None]
    d = dy * gamma
    dx = r[:, None] * (d - xh * (d * xh).mean(axis=1, keepdims=True))
    size = r[:, None] * (np.abs(d) + np.abs(xh) * np.abs(d * xh).mean(axis=1, keepdims=True))
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
        size = size + np.abs(np.asarray(dres, np.float64))
    return dx, (dy * xh).sum(axis=0), size, np.abs(dy * xh).sum(axis=0)


def sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def swiglu_fwd(gate, up):
    gate, up = np.asarray(gate, np.float64), np.asarray(up, np.float64)
    return gate * sigmoid(gate) * up


def swiglu_bwd(dy, gate, up):
    """dgate, dup, and the magnitude of dgate's terms."""
    dy, gate, up = (np.asarray(a, np.float64) for a in (dy, gate, up))
    s = sigmoid(gate)
    return dy * up * s * (1.0 + gate * (1.0 - s)), dy * gate * s, np.abs(dy * up) * s * (1.0 + np.abs(gate))


def dequantize(fmt, codes, scales, texp, rows, k):
    """The float64 values [rows, k] that stored bytes stand for: codes and
    scales are the flat uint8 buffers of a quantized operand."""
    if fmt == FP8:
        v = F.e4m3_decode(codes.reshape(rows, k))
    else:
        blk, kind = FP4_VARIANT[fmt]
        v = F.e2m1_decode(F.unpack_nibbles(codes.reshape(rows, k // 2)))
        if kind == "bf16":
            s = F.bf16_decode(scales.view(np.uint16).reshape(rows, k // blk))
        else:
            s = (F.e4m3_decode if kind == "e4m3" else F.e8m0_decode)(scales.reshape(rows, k // blk))
        v = np.asarray(v, np.float64) * np.repeat(np.asarray(s, np.float64), blk, axis=1)
    e = texp if fmt == FP8 or FP4_VARIANT[fmt][1] == "e4m3" else 0
    return np.ldexp(np.asarray(v, np.float64), e)
