"""Helpers of the tests of the operators around the linear layers.

Tolerances count roundings. U = 2^-24 is half a step of fp32, relative; a
bf16 output adds half a step of its own, 2^-8.
"""
import numpy as np
import torch

import sub_byte_mixed_amd as S
from oracle import quantize as OQ
from parity import compare_codes, gpu_codes, say  # noqa: F401

U = 2.0 ** -24
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}
BF, F32 = torch.bfloat16, torch.float32


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype)


def strided(t, pad=0):
    """t on the GPU as a view of wider rows, the gap filled with a huge value
    that would show in any sum it got into. pad = 0: rows as close as their
    alignment allows."""
    rows, cols = t.shape
    ld = -(-cols // 8) * 8 + pad
    buf = torch.full((rows, ld), 3.0e38, dtype=t.dtype, device="cuda")
    buf[:, :cols] = t.cuda()
    return buf[:, :cols]


class Guarded:
    """An output matrix inside a buffer of a known pattern: `intact` tells
    whether anything but the matrix was written."""

    def __init__(self, rows, cols, dtype, pad=8):
        ld = -(-cols // 8) * 8 + pad
        self.buf = torch.full((rows + 2, ld), 7.0, dtype=dtype, device="cuda")
        self.t = self.buf[1:rows + 1, :cols]

    def intact(self):
        rows, cols = self.t.shape
        b = self.buf.clone()
        b[1:rows + 1, :cols] = 7.0
        return bool((b == 7.0).all())


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def close(got, want, rel, what, size=None, floor=0.0):
    """|got - want| <= rel * size (+ the output type's half step, + floor)."""
    g = f64(got)
    size = np.abs(want) if size is None else size
    tol = rel * size + HALF[got.dtype] * np.abs(want) + floor
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, first at {np.argwhere(bad)[0].tolist()}: "
                           f"{g[bad][0]} for {want[bad][0]} (tolerance {np.broadcast_to(tol, g.shape)[bad][0]})")


def check_quantized(q, stats, y32, fmt, rounding, seed, tid, amax, what):
    """q and stats against the oracle's quantization of the fp32 values that
    the same launch stored: bit for bit."""
    o = OQ.quantize(y32.cpu().numpy(), fmt, {S.RNE: "rne", S.SR: "sr"}[rounding], seed, tid, amax=amax)
    compare_codes(gpu_codes(q), o, fmt, what=what)
    if stats is not None:
        st, so = S.decode_stats(stats)[0], o["stats"]
        assert st["amax"] == float(so["amax"]), what
        assert st["n_nonfinite"] == so["n_nonfinite"], what
        for k in ("sum_err2", "sum_x2"):
            assert abs(st[k] - so[k]) <= 1e-5 * so[k], (what, k, st[k], so[k])
