"""snipop_rmsnorm_fwd / _bwd against the float64 oracle: types, widths next to
every change of the kernels' shapes and to no multiple of anything, strides,
in-place updates, quantized outputs, empty-handed calls, streams, graphs.

Tolerances, U = 2^-24. Forward: one rounding in h, one each in the square, its
sum's additions (at most 16 in a thread, 10 across the wave and the waves:
26 on the whole path), the mean, eps, root and reciprocal, halved by the root,
and two products: below 32 U of |y|, and below 20 U of r. Backward: as many on
the way to the mean of d xh, plus the terms' own: 48 U of the sum of the
terms' magnitudes; dgamma adds rows / 512 + 32 additions of partial sums, 96 U
of its sum of magnitudes at up to 2048 rows a workgroup's share of 4."""
import numpy as np
import pytest
import torch

import sub_byte_mixed_amd as S
from oracle import ops as OO
from ops_common import BF, F32, U, Guarded, check_quantized, close, f64, rand, say, strided

pytestmark = pytest.mark.gpu

EPS = 1e-5
SHAPES = [(1, 1), (1, 2048), (2, 7), (3, 8), (5, 48), (4, 512), (9, 520), (257, 1000), (6, 2048), (3, 2051), (2, 4096),
          (5, 4104), (2, 8192), (3, 8195), (2, 16384)]
TYPES = [(BF, BF, BF), (F32, BF, F32), (BF, F32, BF), (F32, F32, BF), (F32, None, BF), (BF, None, F32)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("xt,rt,gt", TYPES)
def test_forward(rows, cols, xt, rt, gt):
    say("rmsnorm_fwd", rows, cols, xt, rt, gt)
    x = rand((rows, cols), xt, 1)
    res = None if rt is None else rand((rows, cols), rt, 2, 2.0)
    gamma = rand((cols,), gt, 3)
    for yt in (F32, BF):
        h, y = Guarded(rows, cols, yt), Guarded(rows, cols, yt, pad=16)
        _, _, r, _, _ = S.rmsnorm_fwd(strided(x, 8), gamma.cuda(), EPS, res=None if res is None else strided(res, 24),
                                      h=h.t, y=y.t)
        wh, wr, wy = OO.rmsnorm_fwd(f64(x), f64(gamma), EPS, None if res is None else f64(res))
        close(h.t, wh, U, "h")
        close(r, wr, 20 * U, "rstd")
        close(y.t, wy, 32 * U, "y")
        assert h.intact() and y.intact()


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (2, 512), (130, 528), (4, 2048), (3, 4096), (2, 8192), (1, 16384)])
@pytest.mark.parametrize("fmt", [S.FP8, S.NVFP4])
@pytest.mark.parametrize("rounding", [S.RNE, S.SR])
def test_quantized_output(rows, cols, fmt, rounding):
    quantized_output(rows, cols, fmt, rounding)


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (130, 544), (4, 2048), (2, 8192)])
@pytest.mark.parametrize("rounding", [S.RNE, S.SR])
def test_quantized_output_mx(rows, cols, rounding):
    quantized_output(rows, cols, S.MXFP4, rounding)


def quantized_output(rows, cols, fmt, rounding):
    say("rmsnorm_fwd quantized", rows, cols, fmt, rounding)
    x, res = rand((rows, cols), F32, 4), rand((rows, cols), BF, 5, 3.0)
    x[0, :min(16, cols)] = 0.0
    res[0, :min(16, cols)] = 0.0                       # a block of zeros
    gamma = rand((cols,), BF, 6)
    a = [t.cuda() for t in (x, gamma)] + [EPS, res.cuda()]
    y0 = S.rmsnorm_fwd(*a, y_dtype=F32)[0]
    for amax in (None, 2.5, 40.0):
        dev = None if amax is None else torch.tensor([amax], dtype=F32, device="cuda")
        y, h, r, q, st = S.rmsnorm_fwd(*a, y_dtype=F32, out_fmt=fmt, rounding=rounding, seed=77, tensor_id=9, amax=dev)
        assert torch.equal(y, y0)                      # the quantized output changes nothing else
        check_quantized(q, st, y, fmt, rounding, 77, 9, None if amax is None else np.float32(amax), f"amax {amax}")
        # alone, and without statistics: the same bytes
        _, _, _, q2, st2 = S.rmsnorm_fwd(*a, with_y=False, with_rstd=False, out_fmt=fmt, rounding=rounding, seed=77,
                                         tensor_id=9, amax=dev, with_stats=False)
        assert st2 is None and torch.equal(q.codes, q2.codes) and torch.equal(q.texp, q2.texp)
        assert fmt == S.FP8 or torch.equal(q.scales, q2.scales)


def test_quantized_output_is_a_gemm_operand():
    """The codes go straight into qgemm: the same product as of snip_quantize
    on an equal tensor (gamma and rows chosen so that y is exact in bf16)."""
    x = torch.ones((128, 256), dtype=BF, device="cuda")
    x[:, ::2] = -1.0                                   # mean h^2 = 1, eps = 0: y = +-gamma
    gamma = rand((256,), BF, 8).cuda()
    y, _, _, q, _ = S.rmsnorm_fwd(x, gamma, 0.0, out_fmt=S.NVFP4)
    q2, _ = S.quantize(y, S.ROWWISE, S.NVFP4)
    w, _ = S.quantize(rand((64, 256), BF, 9, 0.02).cuda(), S.ROWWISE, S.NVFP4)
    assert torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales) and torch.equal(q.texp, q2.texp)
    assert torch.equal(S.qgemm(q, w), S.qgemm(q2, w))


def test_in_place():
    x, res, gamma = rand((37, 1000), BF, 10).cuda(), rand((37, 1000), BF, 11).cuda(), rand((1000,), F32, 12).cuda()
    y0, h0, r0, _, _ = S.rmsnorm_fwd(x, gamma, EPS, res=res)
    stream = res.clone()
    y1, h1, r1, _, _ = S.rmsnorm_fwd(x, gamma, EPS, res=stream, h=stream)
    assert h1 is stream and torch.equal(stream, h0) and torch.equal(y1, y0) and torch.equal(r1, r0)
    x1 = x.clone()
    S.rmsnorm_fwd(x1, gamma, EPS, res=res, h=x1)
    assert torch.equal(x1, h0)
    # the pass for the maximum reads the inputs before they are overwritten
    gamma, x, res = gamma[:992].contiguous(), x[:, :992].contiguous(), res[:, :992].contiguous()
    q0 = S.rmsnorm_fwd(x, gamma, EPS, res=res, out_fmt=S.FP8)[3]
    stream = res.clone()
    q1 = S.rmsnorm_fwd(x, gamma, EPS, res=stream, h=stream, out_fmt=S.FP8)[3]
    assert torch.equal(q0.codes, q1.codes) and torch.equal(q0.texp, q1.texp)
    dy, dres = rand((37, 992), BF, 13).cuda(), rand((37, 992), BF, 14).cuda()
    rstd = S.rmsnorm_fwd(x, gamma, EPS)[2]
    dx0, dg0 = S.rmsnorm_bwd(dy, x, gamma, rstd, dres=dres)
    g = dres.clone()
    dx1, dg1 = S.rmsnorm_bwd(dy, x, gamma, rstd, dres=g, dx=g)
    assert torch.equal(g, dx0) and torch.equal(dg0, dg1)
    d = dy.clone()
    S.rmsnorm_bwd(d, x, gamma, rstd, dres=dres, dx=d)
    assert torch.equal(d, dx0)


def test_rows_of_zeros_and_nonfinite_rows():
    x = rand((5, 544), BF, 15)
    x[1] = 0.0
    x[2, 3] = float("inf")
    x[3, 500] = float("nan")
    gamma = torch.ones(544, dtype=BF)
    y, _, r, q, st = S.rmsnorm_fwd(x.cuda(), gamma.cuda(), EPS, y_dtype=F32, out_fmt=S.FP8)
    _, wr, wy = OO.rmsnorm_fwd(f64(x)[[0, 1, 4]], f64(gamma), EPS)
    close(y[[0, 1, 4]], wy, 32 * U, "finite rows")
    close(r[[0, 1, 4]], wr, 20 * U, "rstd")
    assert torch.isnan(y[2, 3]) and (y[2, :3] == 0).all() and torch.isnan(y[3]).all()
    s = S.decode_stats(st)[0]
    assert s["n_nonfinite"] == int((~torch.isfinite(y)).sum())
    assert s["amax"] == float(y[torch.isfinite(y)].abs().max())
    # one row of zeros alone, no eps: 1 / 0 is infinite, 0 * inf is NaN, as the formula has it
    y = S.rmsnorm_fwd(torch.zeros((1, 64), dtype=BF, device="cuda"), torch.ones(64, dtype=BF, device="cuda"), 0.0)[0]
    assert torch.isnan(y).all()


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2048), (2, 7), (3, 512), (700, 500), (2000, 2048), (9, 2051),
                                       (33, 4104), (5, 8192), (3, 8195), (2, 16384)])
@pytest.mark.parametrize("yt,ht,rt,gt", [(BF, BF, BF, BF), (F32, BF, BF, BF), (F32, F32, F32, F32), (BF, F32, None, BF),
                                         (F32, BF, None, BF), (BF, BF, F32, BF)])
def test_backward(rows, cols, yt, ht, rt, gt):
    say("rmsnorm_bwd", rows, cols, yt, ht, rt, gt)
    dy, h, gamma = rand((rows, cols), yt, 20), rand((rows, cols), ht, 21, 2.0), rand((cols,), gt, 22)
    dres = None if rt is None else rand((rows, cols), rt, 23)
    r = torch.from_numpy(1.0 / np.sqrt((f64(h) ** 2).mean(1) + EPS)).to(F32)
    want_dx, want_dg, size, gsize = OO.rmsnorm_bwd(f64(dy), f64(h), f64(gamma), f64(r), None if dres is None else f64(dres))
    args = (strided(dy, 8), strided(h, 16), gamma.cuda(), r.cuda())
    for xt in (F32, BF):
        dx = Guarded(rows, cols, xt)
        dg = torch.full((cols + 8,), 5.0, dtype=F32, device="cuda")
        S.rmsnorm_bwd(*args, dres=None if dres is None else strided(dres), dx=dx.t, dgamma=dg[:cols])
        close(dx.t, want_dx, 48 * U, "dx", size=size)
        close(dg[:cols], want_dg, 96 * U, "dgamma", size=gsize)
        assert dx.intact() and (dg[cols:] == 5.0).all()
    # each output alone, and again: the same bits
    only, none = S.rmsnorm_bwd(*args, need_dgamma=False, dx_dtype=BF, dres=None if dres is None else strided(dres))
    assert none is None and torch.equal(only, dx.t)
    none, only = S.rmsnorm_bwd(*args, need_dx=False, dres=None if dres is None else strided(dres))
    assert none is None and torch.equal(only, dg[:cols])


def test_gradient_against_differences():
    """The backward call's gradients against central differences of the
    forward call's y (fp32 throughout). With a step of 2^-6 a difference of
    two sums of 160 terms carries at most 160 * 32 U |y w| / 2^-5 of rounding,
    below 2e-2 here, and (step^2) / 6 of a third derivative that stays below
    30: 1e-3."""
    rows, cols = 5, 32
    x, res, gamma, w = (rand(s, F32, 30 + i) for i, s in enumerate([(rows, cols), (rows, cols), (cols,), (rows, cols)]))

    def loss(x, res, gamma):
        y = S.rmsnorm_fwd(x.cuda(), gamma.cuda(), EPS, res=res.cuda(), y_dtype=F32, h_dtype=F32)[0]
        return float((y.double().cpu() * w.double()).sum())
    _, h, r, _, _ = S.rmsnorm_fwd(x.cuda(), gamma.cuda(), EPS, res=res.cuda(), y_dtype=F32, h_dtype=F32)
    dx, dg = S.rmsnorm_bwd(w.cuda(), h, gamma.cuda(), r, dx_dtype=F32)
    step = 2.0 ** -6
    for t, grad, at in ((0, dx, (2, 5)), (0, dx, (4, 31)), (1, dx, (0, 0)), (1, dx, (3, 17)), (2, dg, (7,)), (2, dg, (30,))):
        a, b = [[v.clone() for v in (x, res, gamma)] for _ in range(2)]
        a[t][at] += step
        b[t][at] -= step
        d = (loss(*a) - loss(*b)) / (2 * step)
        assert abs(d - float(grad[at])) < 2e-2, (t, at, d, float(grad[at]))


def test_long_batch_passes_32_bit_offsets():
    """More than 2^31 elements of a matrix: the last rows against themselves
    in a small call."""
    rows, cols = 131136, 16384
    x = torch.zeros((rows, cols), dtype=BF, device="cuda")
    tail = rand((3, cols), BF, 40).cuda()
    x[-3:] = tail
    gamma = rand((cols,), BF, 41).cuda()
    _, _, r, q, _ = S.rmsnorm_fwd(x, gamma, EPS, with_y=False, h=x, out_fmt=S.FP8,
                                  amax=torch.tensor([8.0], device="cuda"), with_stats=False)
    _, _, r2, q2, _ = S.rmsnorm_fwd(tail, gamma, EPS, with_y=False, out_fmt=S.FP8,
                                    amax=torch.tensor([8.0], device="cuda"), with_stats=False)
    assert torch.equal(r[-3:], r2) and torch.equal(x[-3:], tail)
    assert torch.equal(q.codes[-3 * cols:], q2.codes) and not (q.codes[:-3 * cols] & 0x7F).any()   # zeros take gamma's sign


def test_other_stream():
    x, gamma = rand((300, 2048), BF, 50).cuda(), rand((2048,), BF, 51).cuda()
    y0, _, r0, q0, st0 = S.rmsnorm_fwd(x, gamma, EPS, out_fmt=S.NVFP4)
    dx0, dg0 = S.rmsnorm_bwd(y0, x, gamma, r0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle in (side, side.cuda_stream):
        y, _, r, q, st = S.rmsnorm_fwd(x, gamma, EPS, out_fmt=S.NVFP4, stream=handle)
        dx, dg = S.rmsnorm_bwd(y, x, gamma, r, stream=handle)
        side.synchronize()
        assert torch.equal(y, y0) and torch.equal(q.codes, q0.codes) and torch.equal(st, st0)
        assert torch.equal(dx, dx0) and torch.equal(dg, dg0)


@pytest.mark.parametrize("rows,cols", [(7, 513), (300, 520), (41, 777), (1030, 1008), (9, 1024), (3, 1025)])
@pytest.mark.parametrize("xt,rt,gt", [(BF, F32, BF), (F32, None, F32)])
def test_widths_of_two_chunks_a_lane(rows, cols, xt, rt, gt):
    """Rows that a wave holds in two chunks a lane, and the width just beyond."""
    test_forward(rows, cols, xt, rt, gt)
    test_backward(rows, cols, xt, BF, rt, gt)
    test_backward(rows, cols, xt, F32, rt, gt)
