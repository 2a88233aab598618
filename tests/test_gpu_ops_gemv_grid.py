"""snipop_qgemv with more row tiles than one row of a grid holds."""
import pytest
import torch

import sub_byte_mixed_amd as S
from ops_common import BF, rand, say
from test_gpu_ops_gemv import check, raw_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n", [(2, (1 << 30) + 5), (5, (1 << 26) + 121)])
def test_more_tiles_than_a_grid_row(m, n):
    """Zeros (of 2^30 rows and more), but for rows on both sides of the tile at
    which the grid's second row starts, and the last ones."""
    k, few, rt = 32, 27, 1 if m <= 4 else 4
    w = S.QuantizedTensor(S.MXFP4, n, k, "cuda")
    w.codes.zero_()
    w.scales.zero_()
    small = raw_weights(S.MXFP4, few, k, 21)
    starts = ((1 << 20) * 16 * rt - 13, n - few)
    for at in starts:
        w.codes.view(n, k // 2)[at:at + few] = small.codes.view(few, k // 2)
        w.scales[at:at + few] = small.scales
    x = rand((m, k), BF, 22).cuda()
    say("gemv grid", n, m)
    y = S.qgemv(x, w, y_dtype=BF)
    for at in starts:
        check(x, small, y[:, at:at + few])
        y[:, at:at + few] = 0
    assert not y.any()
