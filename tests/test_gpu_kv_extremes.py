"""snipkv_attn at the ends of what its arguments may be, in the launch for few
rows (a workgroup a unit, and steps shared among workgroups) and in the one for
prompts (eight and four waves a workgroup), against float64 as in
test_gpu_kv_attn.py."""
import numpy as np
import pytest
import torch

import sub_byte_mixed_amd as S
from kv_common import Paged
from ops_common import BF, rand, say

pytestmark = pytest.mark.gpu
FORMATS = [S.NVFP4, S.MXFP4]
UNIT = {64: 128, 128: 128, 256: 64}                    # rows of a workgroup for prompts
LAUNCHES = {"whole": 0, "shared": 0, "eight": 256, "four": 1024}     # units that a call of prompts has at least


def paged(launch, fmt, dim, group, seed, keys=0, **more):
    """One sequence for a launch: three new tokens of `keys` (100 where 0), or a prompt of 600, after 40 others."""
    if LAUNCHES[launch]:
        new = 600
        heads = -(-LAUNCHES[launch] // (new * group // UNIT[dim]))
        return Paged(fmt, dim, heads, 16, [keys or new + 40], [new], seed=seed, **more)
    return Paged(fmt, dim, 2, 16, [keys or 100], [3], seed=seed, capacity=5000 if launch == "shared" else 0, **more)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("launch", LAUNCHES)
@pytest.mark.parametrize("far,window", [
    (2 ** 31 - 1, 2 ** 30),                            # the window lies behind the table: no key
    (2 ** 30 + 500, 2 ** 30),                          # some rows' reaches into it
    (2 ** 31 - 1, 2 ** 31 - 201),
    (2 ** 31 - 1, 2 ** 31 - 1),                        # all of it
    (2 ** 31 - 1, 2 ** 31),
])
def test_positions_and_windows_up_to_31_bits(fmt, launch, far, window):
    """lens far behind a short table: rows see the table's keys that their window reaches, or none."""
    say("far", fmt, launch, far, window)
    P = paged(launch, fmt, 64, 2, 31, 704)             # pages are full
    q = rand((P.rows, P.heads * 2 * 64), BF, 1, 0.5)
    P.batch.lens.fill_(far)
    P.positions = lambda b: far - P.new[b] + np.arange(P.new[b], dtype=np.int64)
    out, lse = S.kv_attn(q.cuda(), P.cache, P.batch, window=window, with_lse=True)
    P.check(q, out, lse, None, window)
    if (far, window) == (2 ** 31 - 1, 2 ** 30):
        assert not out.any() and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("launch", LAUNCHES)
@pytest.mark.parametrize("scale", [1e-36, 1e-38, 1e-40])
def test_scales_far_below_one(launch, scale):
    """MXFP4's keys times queries up to 2^127 under a scale that brings them back."""
    scale = float(np.float32(scale))
    say("small scale", launch, scale)
    P = paged(launch, S.MXFP4, 64, 2, 32)
    t = P.cache.k_scales
    new = torch.randint(127 + 50, 127 + 58, t.shape, generator=torch.Generator().manual_seed(1), dtype=torch.uint8).cuda()
    t.copy_(torch.where(t == 0xFF, t, new))
    q = rand((P.rows, P.heads * 2 * 64), torch.float32, 2).clamp(-4, 4).mul(2.0 ** 60).to(BF)
    out, lse = S.kv_attn(q.cuda(), P.cache, P.batch, scale=scale, with_lse=True)
    P.check(q, out, lse, scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("launch", LAUNCHES)
def test_queries_with_dimensions_far_below_their_largest(fmt, dim, launch):
    """A query's largest dimension meets keys of zero; the score comes from dimensions of 2^-17 of it, which are held
    exactly. So the results and tolerances are those of queries without the largest."""
    say("small dimensions", fmt, dim, launch)
    P = paged(launch, fmt, dim, 2, 33)
    P.cache.k_codes[:, :, :, 0, :, 0] &= 0xF0          # dimension 0
    g = torch.Generator().manual_seed(3)
    small = torch.zeros((P.rows, P.heads * 2, dim))
    small[:, :, 1:32] = 2.0 ** -17 * (1.0 + 2.0 ** -7) * (2.0 * torch.randint(0, 2, (P.rows, P.heads * 2, 31), generator=g) - 1.0)
    q = small.clone()
    q[:, :, 0] = 1.0
    q, small = (t.reshape(P.rows, -1).to(BF) for t in (q, small))
    scale = 2.0 ** (15 if fmt == S.NVFP4 else 14)
    out, lse = S.kv_attn(q.cuda(), P.cache, P.batch, scale=scale, with_lse=True)
    P.check(small, out, lse, scale)


def check(P, q, scale=None, window=0):
    out, lse = S.kv_attn(q.cuda(), P.cache, P.batch, scale=scale, window=window, with_lse=True)
    P.check(q, out, lse, scale, window)
    again, _ = S.kv_attn(q.cuda(), P.cache, P.batch, scale=scale, window=window)
    assert torch.equal(again, out)
    return out, lse


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("launch", ["eight", "four"])
@pytest.mark.parametrize("qscale,scale", [(0.0, None), (40.0, None), (1e-30, 1e29), (1e30, 1e-30), (0.5, 3.0)])
def test_sizes_of_scores(fmt, launch, qscale, scale):
    """Queries of zero; peaked softmaxes; queries far from 1 under a scale that brings them back."""
    say("prompt sizes", fmt, launch, qscale, scale)
    P = paged(launch, fmt, 64, 2, 7)
    check(P, rand((P.rows, P.heads * 2 * 64), BF, 1, qscale), scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("launch", ["eight", "four"])
def test_rising_scores(fmt, dim, launch):
    """Keys whose scores grow along the sequence: the running maximum moves from tile to tile."""
    say("prompt rising", fmt, dim, launch)
    P = paged(launch, fmt, dim, 2, 8)
    base, step = (0x20, 8) if fmt == S.NVFP4 else (118, 1)
    t = P.cache.k_scales.transpose(3, 4)
    for j in range(0, P.lens[0], 16):
        up = torch.arange(j, j + min(16, P.lens[0] - j)) // 90
        t[int(P.table[0, j // 16]), :, 0, :len(up)] = (base + step * up[:, None, None]).to(torch.uint8).cuda()
    check(P, rand((P.rows, P.heads * 2 * dim), BF, 1, 0.5))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("launch", ["eight", "four"])
def test_queries_that_are_not_finite(fmt, launch):
    """They reach their own rows alone."""
    say("prompt, not finite", fmt, launch)
    P = paged(launch, fmt, 128, 2, 9)
    q = rand((P.rows, P.heads * 2 * 128), BF, 5, 0.5)
    odd = q.clone()
    bad = [(3, 0, 7), (3, 2, 100), (300, 1, 0), (599, 3, 127), (64, 0, 64), (65, 0, 1)]      # token, head, dimension
    for i, (t, h, d) in enumerate(bad):
        odd[t, h * 128 + d] = (float("nan"), float("inf"), -float("inf"))[i % 3]
    out, lse = S.kv_attn(odd.cuda(), P.cache, P.batch, with_lse=True)
    want, want_lse = S.kv_attn(q.cuda(), P.cache, P.batch, with_lse=True)
    for t, h, d in bad:
        assert bool(out[t, h * 128:(h + 1) * 128].isnan().all())
        out[t, h * 128:(h + 1) * 128] = want[t, h * 128:(h + 1) * 128]
        lse[t, h] = want_lse[t, h]
    P.check(q, out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("units", [256, 1024])
@pytest.mark.parametrize("window", [0, 33])
def test_prompts_drafts_and_tokens(fmt, dim, units, window):
    """Prompts, chunks after others, drafted and single tokens, none, a page that is not mapped: both launches."""
    lens, new = [333, 40, 170, 250, 9, 1, 90, 700], [333, 40, 131, 4, 0, 1, 65, 33]
    heads = -(-units // (sum(new) * 4 // UNIT[dim]))
    say("mixed", fmt, dim, units, window)
    P = Paged(fmt, dim, heads, 32, lens, new, seed=dim + window, unmapped=[(0, 1), (7, 20)])
    check(P, rand((P.rows, heads * 4 * dim), BF, 1, 0.5), None, window)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("launch", LAUNCHES)
@pytest.mark.parametrize("texp", [-112, -120, -126])
def test_values_far_below_one(dim, launch, texp):
    """A power of two of NVFP4's values is one of the output: bit for bit, down to the smallest normal numbers."""
    say("small values", dim, launch, texp)
    P = paged(launch, S.NVFP4, dim, 2, 34)
    q = rand((P.rows, P.heads * 2 * dim), BF, 4, 0.5).cuda()
    P.cache.texp[1] = 0
    want = S.kv_attn(q, P.cache, P.batch)[0].float()
    P.cache.texp[1] = texp
    got = S.kv_attn(q, P.cache, P.batch)[0].float()
    normal = want.abs() >= 2.0 ** (-126 - texp)
    assert normal.float().mean() > 0.05 and torch.equal(got[normal], torch.ldexp(want, torch.tensor(float(texp), device="cuda"))[normal])
