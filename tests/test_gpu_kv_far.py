"""snipkv_attn where a call of prompts has sequences of few rows and many keys,
which its launch for few rows shares among workgroups: 17 to 64 rows a kv head
with more than 1024 keys. Against float64 as in test_gpu_kv_attn.py."""
import pytest
import torch

import sub_byte_mixed_amd as S
from kv_common import Paged
from ops_common import BF, rand, say

pytestmark = pytest.mark.gpu
FORMATS = [S.NVFP4, S.MXFP4]
UNIT = {64: 128, 128: 128, 256: 64}                    # rows of a workgroup for prompts


def mixed(fmt, dim, group, lens, new, seed):
    heads = -(-256 // (sum(new) * group // UNIT[dim]))
    return Paged(fmt, dim, heads, 32, lens, new, seed=seed)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 900, 1500])
def test_drafts_of_long_sequences_among_prompts(fmt, dim, window):
    """Drafts on both sides of the limits on rows and on keys; a window that leaves few of the keys."""
    group = 8
    lens = [260, 3000, 1024, 1025, 1056, 1057, 2000, 2500, 1, 1400]
    new = [260, 4, 4, 4, 4, 4, 9, 2, 1, 8]
    say("far drafts", fmt, dim, window)
    P = mixed(fmt, dim, group, lens, new, seed=dim + window)
    q = rand((P.rows, P.heads * group * dim), BF, 1, 0.5)
    out, lse = S.kv_attn(q.cuda(), P.cache, P.batch, window=window, with_lse=True)
    P.check(q, out, lse, None, window)
    assert torch.equal(S.kv_attn(q.cuda(), P.cache, P.batch, window=window)[0], out)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_draft_of_a_long_sequence_is_shared(fmt, dim):
    """Beside a prompt its steps go to many workgroups, each of which leaves its part in the workspace; walked by one
    workgroup a unit, 65536 keys took 13 times as long."""
    P = mixed(fmt, dim, 8, [300, 6000], [300, 4], seed=dim)
    q = rand((P.rows, P.heads * 8 * dim), BF, 2, 0.5)
    ws = torch.full((S.lib().snipkv_attn_workspace(P.rows, 2, P.heads * 8, P.heads, dim),), 255, dtype=torch.uint8, device="cuda")
    out, lse = S.kv_attn(q.cuda(), P.cache, P.batch, with_lse=True, ws=ws)
    P.check(q, out, lse)
    slots = ws[:512 * 2 * 16 * (dim + 2) * 4].view(-1, 16 * (dim + 2) * 4)     # of the first 512 workgroups, two each
    assert int((slots != 255).any(dim=1).sum()) > 256


def test_graph_replays_follow_the_limits():
    """One captured call whose sequences move from one launch to the other: every replay equals the eager call."""
    P = mixed(S.NVFP4, 128, 8, [400, 2000, 1500], [400, 8, 8], seed=5)
    q = rand((P.rows, P.heads * 8 * 128), BF, 3, 0.5).cuda()
    ws = torch.empty(S.lib().snipkv_attn_workspace(P.rows, 3, P.heads * 8, P.heads, 128), dtype=torch.uint8, device="cuda")
    S.kv_attn(q, P.cache, P.batch, ws=ws)
    torch.cuda.synchronize()
    graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(q)
    with torch.cuda.graph(graph):
        S.kv_attn(q, P.cache, P.batch, ws=ws, out=out)
    for i, (lens, new) in enumerate([((400, 2000, 1500), (400, 8, 8)), ((400, 1000, 1030), (400, 8, 8)), ((400, 2000, 1500), (398, 9, 9)),
                                     ((400, 1024, 1057), (300, 3, 7)), ((8, 2000, 0), (8, 8, 0)), ((400, 2000, 1500), (400, 8, 8))]):
        say("far graph", i)
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
