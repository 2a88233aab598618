"""snipop_qgemv, one token over more rows than waves, where a row is one step
of the walk: more than half of a wave's load and no more than one of it (K of
1025 to 2048 with 4-bit weights, 513 to 1024 in FP8), so that every step turns
to the next row. Against float64 within the library's bar for GEMM outputs."""
import pytest
import torch

import sub_byte_mixed_amd as S
from ops_common import BF, rand, say
from test_gpu_ops_gemv import FORMATS, check, raw_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,k", [(6145, 1056), (6152, 1504), (20011, 2048), (32000, 2048)])
def test_rows_of_one_step(fmt, n, k):
    if fmt == S.FP8:
        k = max(544, k // 64 * 32)                     # half as many weights a load: 544, 736, 1024
    say("gemv one step a row", S.FORMAT_NAMES[fmt], n, k)
    w = raw_weights(fmt, n, k, n + k)
    x = rand((1, k), BF, 71).cuda()
    y = S.qgemv(x, w)
    check(x, w, y)
    assert torch.equal(y, S.qgemv(x, w)) and torch.equal(S.qgemv(x, w, y_dtype=BF), y.to(BF))
