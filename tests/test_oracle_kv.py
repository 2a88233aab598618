"""Pins of oracle/kv.py: the cache's layout index by index, the rotation against
complex numbers, stored values against hand-decoded bytes, attention against a
loop and closed forms."""
import math

import numpy as np
import pytest

from oracle import kv as OK
from oracle.quantize import MXFP4, NVFP4
from sub_byte_mixed_amd import kv as KV

BLOCK = {NVFP4: 16, MXFP4: 32}


@pytest.mark.parametrize("fmt", [NVFP4, MXFP4])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_layout(fmt, dim):
    """Byte i of a token in a buffer filled with its own indices, by the header's formulas."""
    pages, heads, page = 2, 3, 32
    p = 8 if dim == 64 else 16
    s, v = max(1, 2 * p // BLOCK[fmt]), p // 4
    for which, (shape, keys, piece, group) in enumerate(zip(KV.cache_shapes(fmt, pages, page, heads, dim), (True, True, False, False),
                                                            (p, s, v, 1), (16, 16, 4, 4))):
        n = int(np.prod(shape))
        flat = np.arange(n)
        got = OK.token_major(flat.reshape(shape), keys)
        size = dim // 2 if which % 2 == 0 else dim // BLOCK[fmt]
        assert got.shape == (pages, heads, page, size)
        for pg, h, t, b in [(0, 0, 0, 0), (1, 2, 31, size - 1), (0, 1, 17, size // 2), (1, 0, 5, min(size - 1, 3)), (1, 2, 16, 1)]:
            at = ((pg * heads + h) * page + t // group * group) * size + b // piece * group * piece + t % group * piece + b % piece
            assert got[pg, h, t, b] == at


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [8, 4])
def test_rotation(inter, rot):
    g = np.random.default_rng(1)
    x = g.standard_normal((5, 2, 8)).astype(np.float32)
    ang = g.uniform(0, 7, (5, rot // 2))
    y = OK.rotate(x, np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32), inter)
    half = rot // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * ang[:, None, i])
        assert np.abs(y[..., a] - z.real).max() < 4e-7 * 8 and np.abs(y[..., b] - z.imag).max() < 4e-7 * 8
    assert np.array_equal(y[..., rot:], x[..., rot:])
    one = OK.rotate(x, np.ones((5, half), np.float32), np.zeros((5, half), np.float32), inter)
    assert np.array_equal(one, x)


def test_values():
    codes = np.array([[[0x21, 0x43, 0x65, 0x87, 0xA9, 0xCB, 0xED, 0x0F] * 2]], np.uint8)      # nibbles 1, 2, .. 15, 0, twice: 32
    mags = [0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6, 0]
    got = OK.values(NVFP4, codes, np.array([[[0x38, 0x41]]], np.uint8), 3)                      # E4M3 1.0 and 2.25
    assert np.array_equal(got[0, 0], np.concatenate([8.0 * np.array(mags), 18.0 * np.array(mags)]))
    got = OK.values(MXFP4, codes, np.array([[[125]]], np.uint8), 3)                             # 2^-2; no tensor exponent
    assert np.array_equal(got[0, 0], 0.25 * np.array(mags * 2))


def test_attention_against_a_loop():
    g = np.random.default_rng(2)
    rows, heads, dim, n = 4, 2, 6, 9
    q, k, v = g.standard_normal((rows, heads, dim)), g.standard_normal((n, dim)), g.standard_normal((n, dim))
    pos, mapped = np.array([8, 3, -1, 5]), np.array([True] * 4 + [False] * 2 + [True] * 3)
    for window in (0, 3):
        out, lse, size, _, keys = OK.attention(q, k, v, pos, mapped, 0.7, window)
        for r in range(rows):
            for h in range(heads):
                see = [j for j in range(n) if mapped[j] and j <= pos[r] and (not window or j > pos[r] - window)]
                assert keys[r, h] == len(see)
                if not see:
                    assert not out[r, h].any() and lse[r, h] == -math.inf
                    continue
                e = [math.exp(0.7 * float(q[r, h] @ k[j])) for j in see]
                want = sum(w * v[j] for w, j in zip(e, see)) / sum(e)
                assert np.allclose(out[r, h], want, rtol=1e-12, atol=0) and math.isclose(lse[r, h], math.log(sum(e)), rel_tol=1e-12)
                assert np.allclose(size[r, h], sum(w * np.abs(v[j]) for w, j in zip(e, see)) / sum(e))


def test_attention_closed_forms():
    k, v = np.zeros((5, 4)), np.arange(20.0).reshape(5, 4)
    out, lse, *_ = OK.attention(np.ones((1, 1, 4)), k, v, np.array([4]), np.ones(5, bool), 1.0, 0)
    assert np.allclose(out[0, 0], v.mean(axis=0)) and math.isclose(lse[0, 0], math.log(5))
    k[2] = 1000.0                                      # one key takes all
    out, lse, *_ = OK.attention(np.ones((1, 1, 4)), k, v, np.array([4]), np.ones(5, bool), 1.0, 0)
    assert np.array_equal(out[0, 0], v[2]) and lse[0, 0] == 4000.0
