"""snipop_swiglu_fwd quantized from bf16 gate and up, whose chunks are of 8
elements (fp32: 4), with their own stores of codes and scales, lanes of a block
and random draws: bit for bit the oracle's quantization of the fp32 values that
the same launch stored, which are within 8 U of the formula's."""
import numpy as np
import pytest
import torch

import sub_byte_mixed_amd as S
from oracle import ops as OO
from ops_common import BF, F32, U, check_quantized, close, f64, rand, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (130, 544), (4, 5632), (700, 2048)])
@pytest.mark.parametrize("fmt", [S.FP8, S.NVFP4, S.MXFP4])
@pytest.mark.parametrize("rounding", [S.RNE, S.SR])
def test_quantized_output(rows, cols, fmt, rounding):
    say("swiglu_fwd quantized from bf16", rows, cols, fmt, rounding)
    both = rand((rows, 2 * cols), BF, 15, 2.0).cuda()
    g, u = both[:, :cols], both[:, cols:]              # the halves of one product's output
    want = OO.swiglu_fwd(f64(g), f64(u))
    for amax in (None, 3.0):
        dev = None if amax is None else torch.tensor([amax], dtype=F32, device="cuda")
        y, q, st = S.swiglu_fwd(g, u, y_dtype=F32, out_fmt=fmt, rounding=rounding, seed=5, tensor_id=4, amax=dev)
        close(y, want, 8 * U, "y")
        check_quantized(q, st, y, fmt, rounding, 5, 4, None if amax is None else np.float32(amax), f"amax {amax}")
        _, q2, _ = S.swiglu_fwd(g, u, with_y=False, out_fmt=fmt, rounding=rounding, seed=5, tensor_id=4, amax=dev,
                                with_stats=False)
        assert torch.equal(q.codes, q2.codes) and (fmt == S.FP8 or torch.equal(q.scales, q2.scales))
        assert fmt == S.MXFP4 or torch.equal(q.texp, q2.texp)
