"""snipop_qgemv with scales at the ends of their range, E8M0 (2^-127 .. 2^127)
and bf16 (subnormals to the largest), for every number of tokens and tiles a
wave, within the library's bar for GEMM outputs: 1e-5 of sum |a||b|, plus half
a step of bf16 where y is bf16. The tokens are sized so that no result
leaves the normal fp32 numbers."""
import numpy as np
import pytest
import torch

import sub_byte_mixed_amd as S
from ops_common import BF, rand, say
from test_gpu_ops_gemv import check, raw_weights

pytestmark = pytest.mark.gpu

E8M0 = [S.MXFP4, S.FP4_E8M0_B16]
BF16 = [S.FP4_BF16_B16, S.FP4_BF16_B32]
TOP = {"e8m0": (252, 253, 254), "bf16": (0x7DFF, 0x7E00, 0x7ED5, 0x7F00, 0x7F7F)}
BOTTOM = {"e8m0": (0, 1, 2), "bf16": (0x0001, 0x0055, 0x007F, 0x0080, 0x00D5, 0x00FF, 0x0100)}
# N for one to four tiles a wave, ragged last tiles
SHAPES = [(17, 96), (40, 1056), (4117, 288), (12275, 160), (24593, 64)]


def scales_of(w):
    """The scales as [rows][blocks] of their own integer type, on the GPU."""
    t = torch.int16 if S.FP4_LAYOUT[w.format][1] == "bf16" else torch.uint8
    return w.scales.view(t).view(w.rows, -1)


def put(w, row, block, raw):
    s = scales_of(w)
    s[row, block] = torch.tensor(raw, dtype=torch.int32).to(s.dtype).cuda()


@pytest.mark.parametrize("fmt", E8M0 + BF16)
@pytest.mark.parametrize("n,k", SHAPES)
@pytest.mark.parametrize("ends,size", [(TOP, 2.0 ** -40), (BOTTOM, 2.0 ** 40)])
def test_ends_of_the_range(fmt, n, k, ends, size):
    """A few such scales among ordinary ones, in the first and the last tile."""
    w = raw_weights(fmt, n, k, n + k)
    blocks = scales_of(w).shape[1]
    g = np.random.default_rng(k)
    for i, raw in enumerate(ends[S.FP4_LAYOUT[fmt][1]]):
        put(w, i % n, int(g.integers(blocks)), raw)
        put(w, n - 1 - i % n, blocks - 1, raw)
        scales_of(w)[2 * i + 1] = torch.tensor(raw, dtype=torch.int32).to(scales_of(w).dtype).cuda()   # a whole row
    for m in (1, 2, 3, 4, 5, 8, 16):
        say("gemv scales", S.FORMAT_NAMES[fmt], n, k, m, size)
        x = rand((m, k), BF, m, size).cuda()
        y = S.qgemv(x, w)
        check(x, w, y)
        assert torch.equal(S.qgemv(x, w, y_dtype=BF), y.to(BF))


@pytest.mark.parametrize("fmt", E8M0 + BF16)
def test_both_ends_in_one_tile(fmt):
    """Rows whose scales are the largest meet small tokens, rows next to them
    whose scales are the smallest meet large ones: each sees its own alone."""
    n, k = 16, 128
    blk, kind, *_ = S.FP4_LAYOUT[fmt]
    w = raw_weights(fmt, n, k, 3)
    s, codes = scales_of(w), w.codes.view(n, k // 2)
    for row in range(n):
        raw = TOP[kind][-1] if row % 2 else BOTTOM[kind][0]
        s[row] = torch.tensor(raw, dtype=torch.int32).to(s.dtype).cuda()
        codes[row, slice(32, None) if row % 2 else slice(0, 32)] = 0
    for m in (1, 4, 16):
        say("gemv scales, both ends", S.FORMAT_NAMES[fmt], m)
        x = rand((m, k), BF, 90 + m)
        x[:, :64] *= 2.0 ** -40
        x[:, 64:] *= 2.0 ** 40
        check(x.cuda(), w, S.qgemv(x.cuda(), w))


@pytest.mark.parametrize("fmt", E8M0 + BF16)
def test_blocks_of_zeros(fmt):
    """Blocks of zeros (scale 0, or 2^-127 in E8M0) next to ordinary ones, as
    the quantizer writes them, and a row of nothing else."""
    wt = rand((64, 512), BF, 5, 0.02)
    wt[:, 128:192] = 0.0
    wt[7] = 0.0
    w, _ = S.quantize(wt.cuda(), S.ROWWISE, fmt)
    x = rand((16, 512), BF, 6).cuda()
    y = S.qgemv(x, w)
    check(x, w, y)
    assert not y[:, 7].any()
