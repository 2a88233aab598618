"""snipkv_attn with as many rows as its launch for prompts takes (64 row tiles
or more a kv head's sequences), against float64 as in test_gpu_kv_attn.py."""
import math

import pytest
import torch

import sub_byte_mixed_amd as S
from kv_common import Paged, peak
from ops_common import BF, Guarded, rand, say, strided

pytestmark = pytest.mark.gpu
FORMATS = [S.NVFP4, S.MXFP4]
UNIT = {64: 128, 128: 128, 256: 64}                    # rows of a workgroup


def heads_for(dim, rows, units=256):
    """kv heads that give the call the 256 units that the launch is for, or the 1024 of its four waves."""
    return -(-units // (rows // UNIT[dim]))


def run(P, group, window=0, seed=0):
    q = rand((P.rows, P.heads * group * P.dim), BF, seed, 0.5)
    out, lse = S.kv_attn(q.cuda(), P.cache, P.batch, window=window, with_lse=True)
    P.check(q, out, lse, None, window)
    again, _ = S.kv_attn(q.cuda(), P.cache, P.batch, window=window)
    assert torch.equal(again, out)
    return q, out, lse


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 5, 8])
def test_one_prompt(fmt, dim, group):
    new = {1: 2100, 5: 333, 8: 257}[group]
    heads = heads_for(dim, new * group)
    say("prompt", fmt, dim, group, heads)
    run(Paged(fmt, dim, heads, 16, [new + 37], [new], seed=dim + group), group)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,group,new,window", [(64, 8, 135, 0), (64, 5, 410, 100), (128, 16, 130, 0), (128, 3, 700, 33)])
def test_four_waves(fmt, dim, group, new, window):
    heads = heads_for(dim, new * group, 1024)
    say("four waves", fmt, dim, group, heads)
    run(Paged(fmt, dim, heads, 16, [new + 85], [new], seed=dim + group, unmapped=[(0, 3), (0, 8)]), group, window=window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("units", [256, 1024])
@pytest.mark.parametrize("window", [0, 1, 63, 64, 200])
def test_several_sequences(fmt, units, window):
    """Prompts, chunks after others, drafted and single tokens, none: the launch for prompts and that for few rows."""
    lens, new = [700, 40, 250, 333, 9, 1, 90, 1000], [400, 40, 250, 4, 0, 1, 65, 33]
    heads = heads_for(64, sum(new) * 4, units)
    say("prompts", fmt, window, heads)
    run(Paged(fmt, 64, heads, 32, lens, new, seed=window), 4, window=window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_pages_that_are_not_mapped(fmt, dim):
    new = 600
    P = Paged(fmt, dim, heads_for(dim, new * 2), 16, [650], [new], seed=dim, unmapped=[(0, 0), (0, 5), (0, 6), (0, 20), (0, 40)])
    say("prompt, unmapped", fmt, dim)
    run(P, 2)
    run(P, 2, window=30)


def test_rows_of_nobody_and_negative_positions():
    P = Paged(S.NVFP4, 128, heads_for(128, 700 * 2), 16, [500, 100], [600, 100], seed=1)
    q = rand((P.rows + 70, P.heads * 2 * 128), BF, 1)
    out = Guarded(P.rows + 70, P.heads * 256, BF)
    lse = torch.full((P.rows + 70, P.heads * 2), 7.0, device="cuda")
    S.kv_attn(strided(q, 8), P.cache, P.batch, out=out.t, lse=lse)
    P.check(q[:P.rows], out.t, lse)
    assert out.intact() and bool((out.t[P.rows:] == 7.0).all()) and bool((lse[P.rows:] == 7.0).all())
    assert not out.t[:100].any() and bool((lse[:100] == -float("inf")).all())
    d = q.cuda()
    S.kv_attn(d, P.cache, P.batch, out=d)              # in place
    assert torch.equal(d[:P.rows], out.t[:P.rows]) and torch.equal(d[P.rows:].cpu(), q[P.rows:])


def test_many_query_heads_of_one_token():
    """More heads to a kv head than a workgroup has rows, without cu."""
    P = Paged(S.NVFP4, 64, 1, 16, [100 + b for b in range(300)], [1] * 300, one_each=True)
    run(P, 300)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("units", [256, 1024])
def test_many_small_terms(fmt, units):
    """As in test_gpu_kv_attn.py: the part of p keys of 2^-26 of the largest is p 2^-26, off by p 2^-32, the score's
    error of 200 2^-24 times it, and the output's rounding."""
    new = 2100
    P = Paged(fmt, 64, heads_for(64, new, units), 64, [new], [new], seed=22)
    peak(P, 0)
    scale = 26.0 * math.log(2.0) / (64 * (0.125 if fmt == S.NVFP4 else 1.0))
    q = torch.ones((new, P.heads * 64), dtype=BF, device="cuda")
    out, _ = S.kv_attn(q, P.cache, P.batch, scale=scale)
    p = torch.arange(new, dtype=torch.float64)[:, None]
    unit = 2.0 ** -5 if fmt == S.NVFP4 else 1.0
    want = unit * p * 2.0 ** -26 / (1.0 + p * 2.0 ** -26)
    assert bool(((out.cpu().double() - want).abs() <= p * 2.0 ** -32 * unit + want * (2.0 ** -8 + 2.0 ** -11 + 18.1 * 200 * 2.0 ** -24)).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,window", [(64, 100), (128, 17), (256, 100), (64, 0)])
def test_positions_behind_the_table(fmt, dim, window):
    P = Paged(fmt, dim, heads_for(dim, 600 * 2), 16, [650], [600], seed=24, unmapped=[(0, j) for j in range(31, 41)])
    q, out, lse = run(P, 2, window)
    got, z = S.kv_attn(q.cuda(), P.cache, S.KVBatch(P.batch.table[:, :31], P.batch.lens, P.batch.cu), window=window, with_lse=True)
    P.check(q, got, z, None, window)
    if window:
        assert not got[-1].any() and bool((z[-1] == -float("inf")).all())


def test_graph_replays_follow_the_batch():
    """One captured call whose sequences change between prompts, few rows and none: every replay equals the eager call."""
    P = Paged(S.NVFP4, 64, 32, 32, [1100, 900, 700], [500, 200, 100], seed=25)
    q = rand((P.rows, 32 * 4 * 64), BF, 3, 0.5).cuda()
    ws = torch.empty(S.lib().snipkv_attn_workspace(P.rows, 3, 128, 32, 64), dtype=torch.uint8, device="cuda")
    S.kv_attn(q, P.cache, P.batch, ws=ws)
    torch.cuda.synchronize()
    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(graph):
        S.kv_attn(q, P.cache, P.batch, ws=ws, out=out)
    for i, (lens, new) in enumerate([((1100, 900, 700), (500, 200, 100)), ((1100, 33, 5), (790, 9, 1)), ((40, 900, 0), (40, 700, 0)),
                                     ((1, 1, 1), (1, 1, 1)), ((1100, 900, 700), (64, 65, 300)), ((1100, 0, 0), (800, 0, 0))]):
        say("prompt graph", i)
        cu = [0, new[0], new[0] + new[1], sum(new)]
        P.batch.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        P.batch.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        ws.fill_(255)
        out.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = S.kv_attn(q, P.cache, P.batch, out=torch.full_like(q, 7.0))[0]
        assert torch.equal(got, want) and bool((got[cu[3]:] == 7.0).all()), i
