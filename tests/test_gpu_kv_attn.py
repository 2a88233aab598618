"""snipkv_attn against float64 attention over what the cache's bytes stand for.
The cache holds NaN scales wherever no token lies; tolerances are counted in
kv_common.Paged.attention."""
import numpy as np
import pytest
import torch

import sub_byte_mixed_amd as S
from kv_common import Paged, peak
from ops_common import BF, F32, Guarded, f64, rand, say, strided

pytestmark = pytest.mark.gpu
FORMATS = [S.NVFP4, S.MXFP4]
CAPACITIES = [0, 5000]                                 # a workgroup a unit; steps shared among workgroups


def run(P, group, window=0, scale=None, seed=0, qscale=0.5):
    q = rand((P.rows, P.heads * group * P.dim), BF, seed, qscale)
    out, lse = S.kv_attn(q.cuda(), P.cache, P.batch, window=window, scale=scale, with_lse=True)
    P.check(q, out, lse, scale, window)
    again, _ = S.kv_attn(q.cuda(), P.cache, P.batch, window=window, scale=scale)
    assert torch.equal(again, out)
    return q, out, lse


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8, 17])
@pytest.mark.parametrize("capacity", CAPACITIES)
def test_single_tokens(fmt, dim, group, capacity):
    """Lengths around 16, 32, a page and the waves' steps; zero tokens too."""
    say("attn", fmt, dim, group, capacity)
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 200, 0, 300]
    run(Paged(fmt, dim, 2, 16, lens, [1] * len(lens), seed=group, one_each=True, capacity=capacity), group)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [16, 32, 64, 256, 4096])
@pytest.mark.parametrize("capacity", CAPACITIES)
def test_pages(fmt, page, capacity):
    say("attn pages", fmt, page, capacity)
    run(Paged(fmt, 128, 1, page, [page - 1, page, page + 1, 3 * page + 7], [1] * 4, seed=page, one_each=True, capacity=capacity), 4)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 4, 7])
@pytest.mark.parametrize("capacity", CAPACITIES)
def test_prompts_and_tokens(fmt, dim, group, capacity):
    """Whole prompts, chunks after others, drafted tokens, single tokens, no token, in one call."""
    say("attn prompts", fmt, dim, group, capacity)
    lens, new = [45, 100, 67, 300, 1, 50, 161], [45, 37, 1, 4, 1, 0, 130]
    run(Paged(fmt, dim, 2, 32, lens, new, seed=dim + group, capacity=capacity), group)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [1, 2, 16, 31, 32, 100, 2 ** 31 - 1, 2 ** 40])
@pytest.mark.parametrize("capacity", CAPACITIES)
def test_windows(fmt, window, capacity):
    say("attn window", fmt, window, capacity)
    run(Paged(fmt, 64, 2, 16, [5, 200, 333], [5, 70, 1], seed=1, capacity=capacity), 2, window=window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("capacity", CAPACITIES)
def test_pages_that_are_not_mapped(fmt, capacity):
    """Their keys take no part; a row that has none left is zero with lse -inf."""
    P = Paged(fmt, 128, 2, 16, [64, 40, 16, 90], [3, 40, 1, 1], seed=2, unmapped=[(0, 0), (0, 2), (1, 0), (2, 0), (3, 5), (3, 1)],
              capacity=capacity)
    q, out, lse = run(P, 4)
    r = slice(P.cu[1], P.cu[1] + 16)                   # the first page of sequence 1 is all that these see
    assert not out[r].any() and bool((lse[r] == -float("inf")).all())
    assert not out[P.cu[2]].any()
    run(P, 4, window=20)


@pytest.mark.parametrize("capacity", CAPACITIES)
def test_more_new_tokens_than_the_sequence_has(capacity):
    """Rows at negative positions see nothing."""
    P = Paged(S.NVFP4, 64, 1, 16, [5, -3, 0], [9, 2, 4], seed=4, capacity=capacity)
    q, out, lse = run(P, 2)
    assert not out[:4].any() and not out[9:].any() and bool((lse[9:] == -float("inf")).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("length,new,window,wide", [(50, 40, 5, 2), (50, 40, 0, 2), (45, 1, 12, 2), (1500, 300, 50, 81), (1500, 1, 200, 82), (1500, 3, 205, 81)])
def test_positions_behind_the_table(fmt, length, new, window, wide):
    """They see the table's keys that their window reaches, or none."""
    P = Paged(fmt, 64, 2, 16, [length], [new], seed=24, unmapped=[(0, j) for j in range(wide, -(-length // 16))])
    q, out, lse = run(P, 4, window)
    got, z = S.kv_attn(q.cuda(), P.cache, S.KVBatch(P.batch.table[:, :wide], P.batch.lens, P.batch.cu), window=window, with_lse=True)
    P.check(q, got, z, None, window)
    if window and length - window >= 16 * wide:
        assert not got[-1].any() and bool((z[-1] == -float("inf")).all())


@pytest.mark.parametrize("capacity", CAPACITIES)
def test_rows_of_nobody_and_strides(capacity):
    P = Paged(S.NVFP4, 128, 2, 16, [33, 80], [33, 2], seed=5, capacity=capacity)
    q = rand((P.rows + 9, 2 * 2 * 128), BF, 1)
    out = Guarded(P.rows + 9, 512, BF)
    lse = torch.full((P.rows + 9, 4), 7.0, device="cuda")
    S.kv_attn(strided(q, 24), P.cache, P.batch, out=out.t, lse=lse)
    P.check(q[:P.rows], out.t, lse)
    assert out.intact() and bool((out.t[P.rows:] == 7.0).all()) and bool((lse[P.rows:] == 7.0).all())


@pytest.mark.parametrize("capacity", CAPACITIES)
def test_in_place(capacity):
    P = Paged(S.MXFP4, 128, 2, 16, [333, 80], [5, 40], seed=6, capacity=capacity)
    q = rand((P.rows, 512), BF, 1)
    d = q.cuda()
    S.kv_attn(d, P.cache, P.batch, out=d)
    assert torch.equal(d, S.kv_attn(q.cuda(), P.cache, P.batch)[0])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("qscale,scale", [(0.0, None), (40.0, None), (1e-30, 1e29), (1e30, 1e-30), (0.5, 3.0)])
def test_sizes_of_scores(fmt, qscale, scale):
    """Queries of zero; peaked softmaxes; queries far from 1 under a scale that brings them back."""
    say("attn sizes", fmt, qscale, scale)
    run(Paged(fmt, 64, 1, 16, [100, 70], [1, 30], seed=7), 4, scale=scale, qscale=qscale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("capacity", CAPACITIES)
def test_rising_scores(fmt, capacity):
    """Keys whose scores grow along the sequence: the running maximum moves in every tile."""
    P = Paged(fmt, 64, 1, 32, [700], [40], seed=8, capacity=capacity)
    ramp = torch.arange(700) // 90
    base = 0x20 if fmt == S.NVFP4 else 118
    step = 8 if fmt == S.NVFP4 else 1                  # a power of two
    t = P.cache.k_scales.transpose(3, 4)
    for j in range(0, 700, 16):
        n = min(16, 700 - j)
        t[int(P.table[0, j // 32]), :, j % 32 // 16, :n] = (base + step * ramp[j:j + n, None, None]).to(torch.uint8).cuda()
    run(P, 3)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ks,vs", [((0x01, 0x10), (0x70, 0x7F)), ((0x70, 0x7F), (0x01, 0x10)), ((0x00, 0x02), (0x00, 0x02))])
@pytest.mark.parametrize("capacity", CAPACITIES)
def test_scales_at_the_ends(fmt, ks, vs, capacity):
    """E4M3 scales from the subnormal to the largest; E8M0's 2^-127 on, and values to 1e30."""
    if fmt == S.MXFP4:
        ks, vs = [{0x01: (1, 8), 0x70: (125, 135), 0x00: (0, 2)}[a[0]] for a in (ks, vs)]
        vs = (218, 224) if vs == (125, 135) else vs
    P = Paged(fmt, 64, 2, 16, [300, 33], [1, 33], seed=21, capacity=capacity)
    g = torch.Generator().manual_seed(3)
    for t, (lo, hi) in ((P.cache.k_scales, ks), (P.cache.v_scales, vs)):
        new = torch.randint(lo, hi, t.shape, generator=g, dtype=torch.uint8).cuda()
        t.copy_(torch.where(t == (0x7F if fmt == S.NVFP4 else 0xFF), t, new))
    run(P, 4)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("capacity", [0, 30000])
def test_many_small_terms(fmt, dim, capacity):
    """A key that takes nearly all of the softmax and whose value is zero: what is left is the others' part."""
    n = 20000 if capacity else 1200
    P = Paged(fmt, dim, 1, 64, [n], [1], seed=22, capacity=capacity, one_each=True)
    peak(P, n // 3)
    q = torch.ones((1, dim), dtype=BF)
    scale = 26.0 * float(np.log(2.0)) / (dim * (0.125 if fmt == S.NVFP4 else 1.0))
    out, lse = S.kv_attn(q.cuda(), P.cache, P.batch, scale=scale, with_lse=True)
    P.check(q, out, lse, scale)
    assert bool((out.float() > 0.9 * n * 2.0 ** -26 * (2.0 ** -5 if fmt == S.NVFP4 else 1.0)).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("capacity", CAPACITIES)
def test_queries_that_are_not_finite(fmt, capacity):
    """They reach their own rows alone."""
    P = Paged(fmt, 128, 1, 16, [90, 700], [40, 1], seed=23, capacity=capacity)
    q = rand((P.rows, 4 * 128), BF, 5, 0.5)
    odd = q.clone()
    bad = [(3, 0, 7), (3, 2, 100), (17, 1, 0), (39, 3, 127), (40, 0, 64)]      # token, head, dimension
    for i, (t, h, d) in enumerate(bad):
        odd[t, h * 128 + d] = (float("nan"), float("inf"), -float("inf"))[i % 3]
    out, lse = S.kv_attn(odd.cuda(), P.cache, P.batch, with_lse=True)
    want, want_lse = S.kv_attn(q.cuda(), P.cache, P.batch, with_lse=True)
    for t, h, d in bad:
        assert bool(out[t, h * 128:(h + 1) * 128].isnan().all())
        out[t, h * 128:(h + 1) * 128] = want[t, h * 128:(h + 1) * 128]
        lse[t, h] = want_lse[t, h]
    P.check(q, out, lse)


def test_a_key_of_nan_reaches_the_rows_that_see_it():
    P = Paged(S.NVFP4, 64, 1, 16, [40], [40], seed=9)
    P.cache.k_scales.transpose(3, 4)[int(P.table[0, 1]), 0, 0, 4] = 0x7F       # token 20
    q = rand((40, 64), BF, 1)
    out, lse = S.kv_attn(q.cuda(), P.cache, P.batch, with_lse=True)
    assert bool(out[20:].isnan().all()) and bool(lse[20:].isnan().all())
    assert not out[:20].isnan().any() and not lse[:20].isnan().any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,heads,lens,new", [
    (64, 1, [40000], [1]),                             # hundreds of parts to a unit
    (128, 2, [9000, 1500, 1, 3000], [1, 1, 1, 1]),
    (256, 1, [5000, 7000], [1, 1]),
    (128, 1, [6000, 2000, 50], [7, 1, 3]),             # two row tiles
    (64, 3, [3001, 1700], [5, 2]),
])
def test_long_sequences(fmt, dim, heads, lens, new):
    """Many steps to a workgroup, and parts of a unit in many workgroups."""
    say("attn long", fmt, dim, heads, lens)
    P = Paged(fmt, dim, heads, 64, lens, new, seed=10, one_each=max(new) == 1)
    run(P, 8)
    run(P, 5, window=2222)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_cache_larger_than_the_last_level_cache(dim):
    """Its keys are read past that cache."""
    page, heads = 256, 2
    P = Paged(S.NVFP4, dim, heads, page, [3000, 1400], [1, 1], seed=11, one_each=True,
              spare=(130 << 20) // (page * heads * (dim + dim // 8)))
    run(P, 4)
    P = Paged(S.NVFP4, dim, heads, page, [3000, 1400], [6, 1], seed=11, spare=(130 << 20) // (page * heads * (dim + dim // 8)))
    run(P, 4)


@pytest.mark.parametrize("seqs", [65, 700, 5000])
@pytest.mark.parametrize("capacity", CAPACITIES)
def test_many_sequences(seqs, capacity):
    """More than a wave looks up at once, some without tokens, some without new ones."""
    say("attn sequences", seqs, capacity)
    lens = [(37 * b) % 60 for b in range(seqs)]
    run(Paged(S.NVFP4, 64, 1, 16, lens, [1] * seqs, seed=seqs, one_each=True, capacity=capacity), 2)
    run(Paged(S.NVFP4, 64, 1, 16, lens, [min(n, (7 * b) % 3) for b, n in enumerate(lens)], seed=seqs, capacity=capacity), 2)


def test_offsets_past_32_bits():
    """Pages past 4 GiB of codes."""
    fmt, page, heads, dim = S.MXFP4, 256, 8, 256
    per = page * heads * dim // 2
    pages = (5 << 30) // per + 1
    shapes = S.kv.cache_shapes(fmt, pages, page, heads, dim)
    bufs = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in shapes]
    cache = S.KVCache(fmt, *bufs)
    n, use = 2 * page - 9, [pages - 1, pages - 2]
    table = torch.tensor([use], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    k, v, q = (rand((n, heads * dim), BF, i).cuda() for i in range(3))
    S.kv_append(k, v, cache, S.KVBatch(table, lens, cu))
    small = S.KVCache(fmt, *[b[-2:].clone() for b in bufs])
    assert bool(small.k_codes.any()) and bool(small.v_scales.any())
    low = S.KVBatch(torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), lens, cu)
    want, _ = S.kv_attn(q, small, low)
    got, _ = S.kv_attn(q, cache, S.KVBatch(table, lens, cu))
    assert torch.equal(got, want) and bool(want.any())
    assert all(torch.equal(a, b) for a, b in zip(S.kv_gather(cache, S.KVBatch(table, lens, cu), n), S.kv_gather(small, low, n)))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("capacity", CAPACITIES)
def test_what_the_workspace_holds(dim, capacity):
    P = Paged(S.NVFP4, dim, 1, 16, [700, 40], [9, 1], seed=12, capacity=capacity)
    q = rand((P.rows, 4 * dim), BF, 1).cuda()
    want, _ = S.kv_attn(q, P.cache, P.batch)
    ws = torch.empty(S.lib().snipkv_attn_workspace(P.rows, 2, 4, 1, dim) + 256, dtype=torch.uint8, device="cuda")
    for fill in (0, 255, 127):
        ws.fill_(fill)
        got, _ = S.kv_attn(q, P.cache, P.batch, ws=ws[:-256])
        assert torch.equal(got, want) and bool((ws[-256:] == fill).all())


def test_two_calls_at_once():
    """On two streams, each with its own workspace."""
    P = Paged(S.NVFP4, 128, 2, 16, [5000, 3000], [1, 1], seed=13, one_each=True)
    q = [rand((2, 8 * 128), BF, i).cuda() for i in range(2)]
    want = [S.kv_attn(t, P.cache, P.batch)[0] for t in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [S.kv_attn(t, P.cache, P.batch, stream=s)[0] for t, s in zip(q, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
