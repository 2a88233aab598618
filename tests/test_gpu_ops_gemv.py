"""snipop_qgemv against the float64 product of the values that the stored
bytes stand for, within the library's bar for GEMM outputs: 1e-5 of
sum |a||b| (168 roundings of fp32 in a row; a lane sums at most K / 16
products before the 64 lanes and 4 waves join), plus half a step of bf16
where y is bf16."""
import numpy as np
import pytest
import torch

import sub_byte_mixed_amd as S
from oracle import ops as OO
from ops_common import BF, F32, HALF, f64, rand, say

pytestmark = pytest.mark.gpu

FORMATS = [S.FP8, S.NVFP4, S.MXFP4, S.FP4_E4M3_B32, S.FP4_E8M0_B16, S.FP4_BF16_B16, S.FP4_BF16_B32]


def raw_weights(fmt, n, k, seed):
    """Every code, and scales over their range, at random: the bytes of an
    operand as they may come, not only as the quantizer makes them."""
    g = np.random.default_rng(seed)
    w = S.QuantizedTensor(fmt, n, k, "cuda")
    codes = g.integers(0, 256, w.codes.numel(), dtype=np.uint8)
    if fmt == S.FP8:
        codes[(codes & 0x7F) == 0x7F] = 0x7E                          # no NaN
    w.codes.copy_(torch.from_numpy(codes))
    if w.scales is not None:
        kind = S.FP4_LAYOUT[fmt][1]
        m = w.scales.numel()
        if kind == "e4m3":
            sc = g.integers(0, 0x7F, m, dtype=np.uint8)               # zero and subnormal ones too
        elif kind == "e8m0":
            sc = g.integers(110, 140, m, dtype=np.uint8)
        else:
            sc = (2.0 ** g.uniform(-12, 12, m // 2)).astype(np.float32).view(np.uint32) >> 16
            sc = sc.astype(np.uint16).view(np.uint8)
        w.scales.copy_(torch.from_numpy(sc))
    w.texp.fill_(-7)
    return w


def values(w):
    return OO.dequantize(w.format, w.codes.cpu().numpy(), None if w.scales is None else w.scales.cpu().numpy(),
                         int(w.texp.cpu()), w.rows, w.k)


def check(x, w, y):
    a, b = f64(x), values(w)
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = 1e-5 * size + HALF[y.dtype] * np.abs(want)
    bad = ~(np.abs(f64(y) - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), f64(y)[bad][:4], want[bad][:4])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,k", [(1, 32), (5, 64), (17, 96), (256, 2048), (33, 2080), (100, 5632), (16, 8192), (7, 11008)])
def test_formats_and_sizes(fmt, n, k):
    w = raw_weights(fmt, n, k, 7 * n + k)
    for m in (1, 2, 3, 4, 5, 8, 9, 16):
        say("qgemv", fmt, n, k, m)
        x = rand((m, k), BF, m).cuda()
        y = S.qgemv(x, w)
        check(x, w, y)
        assert torch.equal(y, S.qgemv(x, w))                          # the same bits again
        assert torch.equal(S.qgemv(x, w, y_dtype=BF), y.to(BF))


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantizer_output_as_weights(fmt):
    wt = rand((384, 1024), BF, 1, 0.02)
    w, _ = S.quantize(wt.cuda(), S.ROWWISE, fmt)
    x = rand((3, 1024), BF, 2).cuda()
    check(x, w, S.qgemv(x, w))


@pytest.mark.parametrize("m", [1, 3, 7, 16])
def test_strides(m):
    n, k = 70, 320
    w = raw_weights(S.NVFP4, n, k, 3)
    buf = torch.full((m, k + 64), 3.0e38, dtype=BF, device="cuda")
    buf[:, 8:8 + k] = rand((m, k), BF, 4).cuda()
    x = buf[:, 8:8 + k]
    out = torch.full((m + 2, n + 13), 9.0, dtype=F32, device="cuda")
    flat = out.view(-1)[:(m + 1) * (n + 13)]
    y = flat[:m * (n + 13)].view(m, n + 13)[:, :n]                    # odd row stride
    S.qgemv(x, w, y=y)
    check(x, w, y)
    assert torch.equal(y, S.qgemv(x.contiguous(), w))
    rest = out.clone()
    rest.view(-1)[:m * (n + 13)].view(m, n + 13)[:, :n] = 9.0
    assert (rest == 9.0).all()


def test_tokens_do_not_mix():
    """A token's result does not depend on the other tokens' values."""
    w = raw_weights(S.MXFP4, 64, 512, 5)
    for m in (2, 4, 11, 16):
        x = rand((m, 512), BF, 6).cuda()
        y = S.qgemv(x, w)
        x2 = x.clone()
        x2[: m - 1] = float("nan")
        y2 = S.qgemv(x2, w)
        assert torch.equal(y2[m - 1], y[m - 1]) and torch.isnan(y2[: m - 1]).all()


def test_nonfinite_activations():
    w, _ = S.quantize(torch.ones((48, 128), dtype=BF, device="cuda"), S.ROWWISE, S.NVFP4)
    x = torch.ones((2, 128), dtype=BF, device="cuda")
    x[0, 17] = float("inf")
    x[1, 100] = float("nan")
    y = S.qgemv(x, w)
    assert torch.isinf(y[0]).all() and torch.isnan(y[1]).all()


def test_small_and_large_values():
    """bf16 activations over their exponents against weights of 1: no flush
    of small products next to nothing else, no early overflow."""
    w, _ = S.quantize(torch.ones((32, 64), dtype=BF, device="cuda"), S.ROWWISE, S.MXFP4)
    for e in (-100, -60, 0, 60, 100):
        for m in (1, 4, 16):
            x = torch.zeros((m, 64), dtype=BF, device="cuda")
            x[m - 1, 5] = 1.5 * 2.0 ** e
            y = S.qgemv(x, w)
            want = 1.5 * 2.0 ** e
            assert torch.allclose(y[m - 1].double(), torch.full((32,), want, dtype=torch.float64, device="cuda"), rtol=1e-5)


def test_refusals_in_the_binding():
    w = raw_weights(S.NVFP4, 8, 64, 8)
    x = rand((1, 64), BF, 9).cuda()
    with pytest.raises(ValueError):
        S.qgemv(x.float(), w)
    with pytest.raises(ValueError):
        S.qgemv(rand((1, 96), BF, 9).cuda(), w)
    with pytest.raises(ValueError):
        S.qgemv(x, w, y=torch.empty((1, 9), device="cuda"))
    with pytest.raises(S.SnipError) as e:
        S.qgemv(rand((17, 64), BF, 9).cuda(), w)
    assert e.value.code == -2


@pytest.mark.parametrize("fmt", [S.FP8, S.NVFP4, S.MXFP4, S.FP4_BF16_B16])
@pytest.mark.parametrize("n,k", [(8200, 96), (16421, 288), (20, 70016)])
def test_many_rows_and_long_rows(fmt, n, k):
    """The widths at which a wave takes two and four row tiles, and a row too
    long for its scales to be held on chip."""
    w = raw_weights(fmt, n, k, n + k)
    for m in (1, 3, 6, 16):
        say("qgemv", fmt, n, k, m)
        x = rand((m, k), BF, m).cuda()
        check(x, w, S.qgemv(x, w))


@pytest.mark.parametrize("fmt,code", [(S.MXFP4, 255), (S.FP4_E8M0_B16, 255), (S.NVFP4, 0x7F), (S.FP4_E4M3_B32, 0xFF)])
def test_nan_scales_reach_their_row_alone(fmt, code):
    for n, k in ((40, 256), (40, 1056), (8200, 64)):
        w = raw_weights(fmt, n, k, 11)
        sc = w.scales.view(n, -1)
        sc[5, -1] = code
        sc[n - 1, 0] = code
        for m in (1, 4, 16):
            say("nan scale", fmt, n, k, m)
            bad = torch.isnan(S.qgemv(rand((m, k), BF, m).cuda(), w))
            assert bad[:, 5].all() and bad[:, n - 1].all() and int(bad.sum()) == 2 * m


def test_operands_that_do_not_hold_the_weights_are_refused():
    w = raw_weights(S.NVFP4, 8, 64, 8)
    x = rand((1, 64), BF, 9).cuda()
    for bad in (dict(codes=w.codes[:-1]), dict(codes=w.codes.cpu()), dict(scales=w.scales[:-1]), dict(texp=w.texp.cpu())):
        a = dict(codes=w.codes, scales=w.scales, texp=w.texp)
        a.update(bad)
        with pytest.raises(ValueError):
            S.qgemv(x, S.QuantizedTensor(S.NVFP4, 8, 64, "cuda", **a))


@pytest.mark.parametrize("fmt", [S.FP8, S.NVFP4, S.MXFP4, S.FP4_BF16_B16])
@pytest.mark.parametrize("n,k,tokens", [(24593, 64, (4, 7, 16)), (8201, 4128, (1, 2, 3)), (10, 49248, (1, 2)), (4117, 288, (5, 16)), (12275, 160, (5, 16))])
def test_every_form_of_a_launch(fmt, n, k, tokens):
    """Each rule on N, K and the tokens from its other side: many tiles a
    wave, two rows a wave, two tokens in a weight too large for the dot form,
    and a token's values in more than one slab."""
    w = raw_weights(fmt, n, k, n)
    for m in tokens:
        say("gemv forms", S.FORMAT_NAMES[fmt], n, k, m)
        x = rand((m, k), BF, 31 + m).cuda()
        check(x, w, S.qgemv(x, w))


def test_nan_codes_of_fp8_reach_their_row_alone():
    for n, k in ((40, 256), (40, 1056), (8200, 64)):
        w = raw_weights(S.FP8, n, k, 12)
        codes = w.codes.view(n, k)
        codes[3, k - 1], codes[n - 1, 0] = 0x7F, 0xFF
        for m in (1, 2, 4, 16):
            say("nan code", n, k, m)
            bad = torch.isnan(S.qgemv(rand((m, k), BF, m).cuda(), w))
            assert bad[:, 3].all() and bad[:, n - 1].all() and int(bad.sum()) == 2 * m


@pytest.mark.parametrize("m", [1, 3, 16])
def test_weights_beyond_4_gib(m):
    """Rows that start past 2^32 bytes of codes, after rows of zeros."""
    n, k, last = (1 << 19) + 11, 8192 + 32, 27
    w = S.QuantizedTensor(S.FP8, n, k, "cuda")
    w.codes.zero_()
    small = raw_weights(S.FP8, last, k, 13)
    w.codes.view(n, k)[-last:] = small.codes.view(last, k)
    w.texp.copy_(small.texp)
    x = rand((m, k), BF, 60).cuda()
    say("4 GiB", m)
    y = S.qgemv(x, w)
    assert not y[:, :-last].any()
    check(x, small, y[:, -last:])


def test_other_stream():
    w = raw_weights(S.NVFP4, 300, 2048, 14)
    x = rand((4, 2048), BF, 61).cuda()
    want = S.qgemv(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for handle in (side, side.cuda_stream):
        y = S.qgemv(x, w, stream=handle)
        side.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,k", [(6145, 96), (6152, 2080), (20011, 64), (12296, 4128), (6200, 33024)])
def test_rows_that_a_wave_walks(fmt, n, k):
    """One token and more rows than waves: some waves with a row less, rows of
    one chunk and of several, and a token too long to stay on chip."""
    if n * k > 1 << 27 and fmt not in (S.FP8, S.NVFP4):
        pytest.skip("the longest in two formats")
    w = raw_weights(fmt, n, k, n)
    say("gemv walk", S.FORMAT_NAMES[fmt], n, k)
    x = rand((1, k), BF, 62).cuda()
    check(x, w, S.qgemv(x, w))


@pytest.mark.parametrize("fmt,n,k,m", [(S.FP4_BF16_B16, 24593, 14400, 16), (S.NVFP4, 24593, 26112, 7), (S.NVFP4, 4001, 73728, 16),
                                       (S.FP4_BF16_B16, 8209, 33024, 5)])
def test_scales_of_long_rows(fmt, n, k, m):
    """Rows so long that the scales of as many tiles, or beside as many waves,
    as usual do not fit on chip: the first and the last rows of the result."""
    w = S.QuantizedTensor(fmt, n, k, "cuda")
    block, kind, *_ = S.FP4_LAYOUT[fmt]
    per = (k // block) * (2 if kind == "bf16" else 1)
    small = raw_weights(fmt, 50, k, 15)
    at = torch.arange(n, device="cuda") % 50                          # row i holds row i % 50
    w.codes.view(n, k // 2).copy_(small.codes.view(50, k // 2)[at])
    w.scales.view(n, per).copy_(small.scales.view(50, per)[at])
    w.texp.copy_(small.texp)
    x = rand((m, k), BF, 63).cuda()
    say("long rows", S.FORMAT_NAMES[fmt], n, k, m)
    y = S.qgemv(x, w)
    check(x, small, y[:, :50])
    assert torch.equal(y, y[:, :50][:, at])
