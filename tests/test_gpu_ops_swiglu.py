"""snipop_swiglu_fwd / _bwd against the float64 oracle.

Tolerances, U = 2^-24: exp within 2 U, 1 + e and the quotient one rounding
each, the products two: y and dup below 8 U of themselves. dgate sums s and
g s (1 - s), each with its roundings: below 16 U of |dy u| s (1 + |g|). Where
exp(-g) leaves the range of fp32 (g < -88) s is 0 instead of below 1e-38: a
floor of 1e-36 |dy u|, taken as 1e-34."""
import numpy as np
import pytest
import torch

import sub_byte_mixed_amd as S
from oracle import ops as OO
from ops_common import BF, F32, U, Guarded, check_quantized, close, f64, rand, say, strided

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 5632), (2, 7), (3, 8), (64, 64), (7, 1000), (129, 2051), (3, 11008), (2, 28672)]
FLOOR = 1e-34


def inputs(rows, cols, t, seed):
    g, u = rand((rows, cols), t, seed, 3.0), rand((rows, cols), t, seed + 1, 2.0)
    edge = torch.tensor([0.0, -0.0, 20.0, -20.0, 87.0, -87.0, 90.0, -90.0, 1e4, -1e4]).to(t)[:cols]
    g[0, :edge.numel()] = edge
    return g, u


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("t", [BF, F32])
def test_forward(rows, cols, t):
    say("swiglu_fwd", rows, cols, t)
    g, u = inputs(rows, cols, t, 1)
    want = OO.swiglu_fwd(f64(g), f64(u))
    for yt in (F32, BF):
        y = Guarded(rows, cols, yt)
        S.swiglu_fwd(strided(g, 8), strided(u), y=y.t)
        close(y.t, want, 8 * U, "y", floor=FLOOR)
        assert y.intact()


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (130, 544), (4, 5632), (700, 2048)])
@pytest.mark.parametrize("fmt", [S.FP8, S.NVFP4, S.MXFP4])
@pytest.mark.parametrize("rounding", [S.RNE, S.SR])
def test_quantized_output(rows, cols, fmt, rounding):
    say("swiglu_fwd quantized", rows, cols, fmt, rounding)
    both = rand((rows, 2 * cols), F32, 5, 2.0).cuda()
    g, u = both[:, :cols], both[:, cols:]              # the halves of one product's output
    y0 = S.swiglu_fwd(g, u, y_dtype=F32)[0]
    for amax in (None, 3.0):
        dev = None if amax is None else torch.tensor([amax], dtype=F32, device="cuda")
        y, q, st = S.swiglu_fwd(g, u, y_dtype=F32, out_fmt=fmt, rounding=rounding, seed=3, tensor_id=2, amax=dev)
        assert torch.equal(y, y0)
        check_quantized(q, st, y, fmt, rounding, 3, 2, None if amax is None else np.float32(amax), f"amax {amax}")
        _, q2, _ = S.swiglu_fwd(g, u, with_y=False, out_fmt=fmt, rounding=rounding, seed=3, tensor_id=2, amax=dev,
                                with_stats=False)
        assert torch.equal(q.codes, q2.codes)


def test_nonfinite_inputs_are_counted():
    g, u = rand((4, 64), BF, 7), rand((4, 64), BF, 8)
    u[1, 5], g[2, 7] = float("inf"), float("nan")
    y, q, st = S.swiglu_fwd(g.cuda(), u.cuda(), y_dtype=F32, out_fmt=S.NVFP4)
    s = S.decode_stats(st)[0]
    assert s["n_nonfinite"] == 2 and s["amax"] == float(y[torch.isfinite(y)].abs().max())


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt,t", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
def test_backward(rows, cols, dt, t):
    say("swiglu_bwd", rows, cols, dt, t)
    g, u = inputs(rows, cols, t, 11)
    dy = rand((rows, cols), dt, 13)
    wg, wu, size = OO.swiglu_bwd(f64(dy), f64(g), f64(u))
    args = (strided(dy), strided(g, 8), strided(u, 16))
    for ot in (F32, BF):
        dg, du = Guarded(rows, cols, ot), Guarded(rows, cols, ot, pad=16)
        S.swiglu_bwd(*args, dgate=dg.t, dup=du.t)
        close(dg.t, wg, 16 * U, "dgate", size=size, floor=FLOOR)
        close(du.t, wu, 8 * U, "dup", floor=FLOOR)
        assert dg.intact() and du.intact()
    a, none = S.swiglu_bwd(*args, need_dup=False)
    none2, b = S.swiglu_bwd(*args, need_dgate=False)
    assert none is None and none2 is None and torch.equal(a, dg.t) and torch.equal(b, du.t)


def test_in_place():
    g, u, dy = (rand((50, 1000), BF, 20 + i).cuda() for i in range(3))
    y0 = S.swiglu_fwd(g, u)[0]
    a = g.clone()
    assert S.swiglu_fwd(a, u, y=a)[0] is a and torch.equal(a, y0)
    a, b = g.clone(), u.clone()
    dg0, du0 = S.swiglu_bwd(dy, g, u)
    S.swiglu_bwd(dy, a, b, dgate=a, dup=b)
    assert torch.equal(a, dg0) and torch.equal(b, du0)
    g, u = g[:, :992].contiguous(), u[:, :992].contiguous()
    y0, q0, _ = S.swiglu_fwd(g, u, out_fmt=S.FP8)
    a = u.clone()
    _, q1, _ = S.swiglu_fwd(g, a, y=a, out_fmt=S.FP8)  # the pass for the maximum writes nothing
    assert torch.equal(a, y0) and torch.equal(q0.codes, q1.codes)


def test_gradient_against_differences():
    """Central differences of the forward call, step 2^-6: rounding 8 U |y| /
    2^-6 below 1e-4, third derivatives below 2 |u|, times step^2 / 6: 1e-3."""
    g, u, dy = (rand((4, 48), F32, 30 + i) for i in range(3))
    dg, du = S.swiglu_bwd(dy.cuda(), g.cuda(), u.cuda(), dtype=F32)
    step = 2.0 ** -6

    def y(g, u):
        return f64(S.swiglu_fwd(g.cuda(), u.cuda(), y_dtype=F32)[0])
    ng = (y(g + step, u) - y(g - step, u)) / (2 * step) * f64(dy)
    nu = (y(g, u + step) - y(g, u - step)) / (2 * step) * f64(dy)
    lim = 2e-3 * (1.0 + np.abs(f64(u))) * (1.0 + np.abs(f64(dy)))
    assert (np.abs(ng - f64(dg)) < lim).all() and (np.abs(nu - f64(du)) < lim).all()


def test_long_batch_passes_32_bit_offsets():
    """More than 2^31 elements of a matrix: the last rows against themselves
    in a small call, forward and backward, in place to save memory."""
    rows, cols = 195105, 11008
    g, u = (torch.zeros((rows, cols), dtype=BF, device="cuda") for _ in range(2))
    tg, tu, td = (rand((3, cols), BF, 70 + i).cuda() for i in range(3))
    g[-3:], u[-3:] = tg, tu
    say("swiglu", rows, cols)
    _, q, _ = S.swiglu_fwd(g, u, with_y=False, out_fmt=S.FP8, amax=torch.tensor([8.0], device="cuda"), with_stats=False)
    _, q2, _ = S.swiglu_fwd(tg, tu, with_y=False, out_fmt=S.FP8, amax=torch.tensor([8.0], device="cuda"),
                            with_stats=False)
    assert torch.equal(q.codes[-3 * cols:], q2.codes) and not q.codes[:-3 * cols].any()
    dy = torch.ones((rows, cols), dtype=BF, device="cuda")
    dy[-3:] = td
    say("swiglu_bwd", rows, cols)
    S.swiglu_bwd(dy, g, u, dgate=g, dup=u)
    dg, du = S.swiglu_bwd(td, tg, tu)
    assert torch.equal(g[-3:], dg) and torch.equal(u[-3:], du) and not g[:-3].any() and not u[:-3].any()


def test_other_stream():
    g, u, dy = (rand((300, 2048), F32, 80 + i).cuda() for i in range(3))
    y0, q0, st0 = S.swiglu_fwd(g, u, out_fmt=S.MXFP4)
    dg0, du0 = S.swiglu_bwd(dy, g, u)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle in (side, side.cuda_stream):
        y, q, st = S.swiglu_fwd(g, u, out_fmt=S.MXFP4, stream=handle)
        dg, du = S.swiglu_bwd(dy, g, u, stream=handle)
        side.synchronize()
        assert torch.equal(y, y0) and torch.equal(q.codes, q0.codes) and torch.equal(st, st0)
        assert torch.equal(dg, dg0) and torch.equal(du, du0)
