"""The attention half of a block (sub_byte_mixed_amd/attn.py): append, attention
and the products together, for prompts and decode steps; and the calls captured
in HIP graphs whose replays follow the batch's buffers."""
import numpy as np
import pytest
import torch

import sub_byte_mixed_amd as S
from oracle import ops as OO
from sub_byte_mixed_amd.attn import CachedAttention, angles
from ops_common import BF, F32, f64, rand, say

pytestmark = pytest.mark.gpu
HIDDEN, HQ, HK, DIM = 256, 8, 2, 64


def make(fmt=S.NVFP4, pages=40, page=16):
    w = [(1.0 + 0.1 * rand((HIDDEN,), F32, 1)).to(BF), rand(((HQ + 2 * HK) * DIM, HIDDEN), BF, 2, 0.08), rand((HIDDEN, HQ * DIM), BF, 3, 0.05)]
    att = CachedAttention(*[t.cuda() for t in w], HK, DIM, *angles(300, DIM), fmt)
    return w, att, S.KVCache.empty(fmt, pages, page, HK, DIM, "cuda", texp=(-6, -6))


def int32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def weights(q):
    return OO.dequantize(q.format, q.codes.cpu().numpy(), q.scales.cpu().numpy(), int(q.texp.cpu()), q.rows, q.k)


def off(got, want):
    return float(np.linalg.norm(f64(got) - want) / np.linalg.norm(want))


@pytest.mark.parametrize("fmt", [S.NVFP4, S.MXFP4])
def test_decode_steps(fmt):
    """Steps of three sequences, against float64 with the weights that the codes stand for and the keys and values
    that the cache holds. What is left are bf16 roundings of y, q and the attention's output, 2^-8 each at most of
    long sums' terms: 2^-6 of the output bounds them."""
    w, att, cache = make(fmt)
    table = torch.randperm(39, generator=torch.Generator().manual_seed(0))[:30].int().view(3, 10).cuda()
    wqkv, wo = weights(att.q_qkv), weights(att.q_o)
    gamma, cos, sin = f64(w[0]), f64(att.cos), f64(att.sin)
    for step in range(20):
        lens = [step + 1, step + 17, step + 100]
        batch = S.KVBatch(table, int32(*lens))
        x, res = rand((3, HIDDEN), BF, 50 + step), rand((3, HIDDEN), BF, 90 + step)
        if step == 0:                                  # what the longer sequences hold already
            for b in (1, 2):
                n = lens[b] - 1
                S.kv_append(rand((n, HK * DIM), BF, b).cuda(), rand((n, HK * DIM), BF, b + 9).cuda(), cache,
                            S.KVBatch(table[b:b + 1], int32(n), int32(0, n)))
        stream = res.cuda()
        out = att.decode(x.cuda(), stream, cache, batch)
        h = f64(x) + f64(res)
        y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + 1e-5) * gamma
        qkv = y @ wqkv.T
        o = np.zeros((3, HQ * DIM))
        for b in range(3):
            q = qkv[b, :HQ * DIM].reshape(HQ, DIM)
            z = (q[:, :DIM // 2] + 1j * q[:, DIM // 2:]) * (cos + 1j * sin)[lens[b] - 1]
            q = np.concatenate([z.real, z.imag], axis=1)
            n = lens[b]
            k, v = (f64(t).reshape(n, HK, DIM) for t in S.kv_gather(cache, S.KVBatch(table[b:b + 1], int32(n), int32(0, n)), n))
            for i in range(HQ):
                s = k[:, i // (HQ // HK)] @ q[i] / 8.0
                p = np.exp(s - s.max())
                o[b, i * DIM:(i + 1) * DIM] = p @ v[:, i // (HQ // HK)] / p.sum()
        assert off(out, o @ wo.T) < 2.0 ** -6 and off(stream, h) < 2.0 ** -8, step


def test_decode_equals_the_calls():
    _, att, cache = make()
    x, res = rand((2, HIDDEN), BF, 1).cuda(), rand((2, HIDDEN), BF, 2).cuda()
    batch = S.KVBatch(int32(3, 4, 5, 6).view(2, 2), int32(9, 20))
    y, h, _, _, _ = S.rmsnorm_fwd(x, att.gamma, att.eps, res=res)
    qkv = S.qgemv(y, att.q_qkv)
    a, b = HQ * DIM, (HQ + HK) * DIM
    q = S.kv_append(qkv[:, a:b], qkv[:, b:], cache, batch, q=qkv[:, :a], cos=att.cos, sin=att.sin)
    want = S.qgemv(S.kv_attn(q, cache, batch)[0], att.q_o)
    assert torch.equal(att.decode(x, res, cache, batch), want) and torch.equal(res, h)


@pytest.mark.parametrize("fmt", [S.NVFP4, S.MXFP4])
def test_a_prompt_in_one_call_and_in_chunks(fmt):
    """Two sequences padded to 256 rows, and the second of them in two chunks: the same rows' keys, values and
    outputs, up to the tensor scale that a quantized activation takes from its own rows (NVFP4: a power of two of
    the block scales, exact but for E4M3's subnormal range; MXFP4 has none)."""
    say("prompt", fmt)
    _, att, cache = make(fmt)
    x, res = rand((256, HIDDEN), BF, 1).cuda(), rand((256, HIDDEN), BF, 2).cuda()
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    n = (70, 131)
    out = att.prompt(x, res.clone(), cache, S.KVBatch(table, int32(*n), int32(0, 70, 201)))
    assert not out[201:].any()
    other = make(fmt)[2]
    for a, b in ((0, 70), (70, 150), (150, 201)):
        s = 0 if a == 0 else 1
        xs, rs = (torch.zeros((128, HIDDEN), dtype=BF, device="cuda") for _ in range(2))
        xs[:b - a], rs[:b - a] = x[a:b], res[a:b]
        got = att.prompt(xs, rs, other, S.KVBatch(table[s:s + 1], int32(b - (0, 70)[s]), int32(0, b - a)))
        assert off(got[:b - a], f64(out[a:b])) < 1e-2
    for s in range(2):
        batch = S.KVBatch(table[s:s + 1], int32(n[s]), int32(0, n[s]))
        for p, q in zip(S.kv_gather(cache, batch, n[s]), S.kv_gather(other, batch, n[s])):
            assert off(p, f64(q)) < 1e-2


@pytest.mark.parametrize("wide", [10, 200])
def test_graph_replays_follow_the_batch(wide):
    """One captured decode step (short tables: one launch of attention; long ones: two), replayed with lens, table
    and inputs changed in place, with eager work between: every replay equals the eager call."""
    _, att, cache = make(pages=600)
    table = torch.randperm(600, generator=torch.Generator().manual_seed(0))[:3 * wide].int().view(3, wide).cuda()
    batch = S.KVBatch(table, int32(1, 1, 1))
    x, res = (torch.zeros((3, HIDDEN), dtype=BF, device="cuda") for _ in range(2))
    ws = torch.empty(S.lib().snipkv_attn_workspace(3, 3, HQ, HK, DIM), dtype=torch.uint8, device="cuda")
    att.decode(x, res, cache, batch, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = att.decode(x, res, cache, batch, ws=ws)
    for i in range(6):
        say("graph replay", wide, i)
        lens = int32(1 + i, 30 * i + 2, min(300, 16 * wide) - i)
        xs, rs = rand((3, HIDDEN), BF, 2 * i).cuda(), rand((3, HIDDEN), BF, 2 * i + 1).cuda()
        x.copy_(xs)
        res.copy_(rs)
        batch.lens.copy_(lens)
        table.copy_(table.roll(1, 0))
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got, stream = out.clone(), res.clone()
        stored = S.kv_gather(cache, batch)
        want = att.decode(xs, rs, cache, batch)
        assert torch.equal(got, want) and torch.equal(stream, rs), i
        assert all(torch.equal(a, b) for a, b in zip(stored, S.kv_gather(cache, batch))), i


def test_two_graphs_share_a_workspace():
    """Replayed one after the other on one stream."""
    _, att, cache = make(pages=600)
    table = torch.arange(600, dtype=torch.int32, device="cuda").view(2, 300)
    ws = torch.empty(S.lib().snipkv_attn_workspace(2, 2, HQ, HK, DIM), dtype=torch.uint8, device="cuda")
    k, v = rand((4000, HK * DIM), BF, 1).cuda(), rand((4000, HK * DIM), BF, 2).cuda()
    S.kv_append(k, v, cache, S.KVBatch(table, int32(2100, 1900), int32(0, 2100, 4000)))
    batches = [S.KVBatch(table, int32(2100, 1900)), S.KVBatch(table.flip(0).contiguous(), int32(5, 2000))]
    q = [rand((2, HQ * DIM), BF, 5 + i).cuda() for i in range(2)]
    want = [S.kv_attn(a, cache, b)[0] for a, b in zip(q, batches)]
    graphs, outs = [], []
    for a, b in zip(q, batches):
        S.kv_attn(a, cache, b, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(S.kv_attn(a, cache, b, ws=ws)[0])
        graphs.append(g)
    for i in range(6):
        for t in outs:
            t.zero_()
        graphs[i % 2].replay()
        graphs[1 - i % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), i


def test_launches_are_timed():
    _, att, cache = make(pages=600)
    batch = S.KVBatch(torch.arange(600, dtype=torch.int32, device="cuda").view(1, 600), int32(50))
    q = rand((1, HQ * DIM), BF, 1).cuda()
    S.timing_start(16)
    S.kv_append(q[:, :HK * DIM], q[:, :HK * DIM], cache, batch, q=q)
    S.kv_attn(q, cache, batch)
    S.kv_attn(q, cache, S.KVBatch(batch.table[:, :8], batch.lens))
    S.kv_gather(cache, batch)
    recs, untimed = S.timing_read()
    assert untimed == 0 and [r["kind"] for r in recs] == ["kv_append", "kv_attn", "kv_join", "kv_attn", "kv_append"]
    assert all(r["ms"] > 0 and r["format"] == S.NVFP4 for r in recs)
    assert recs[0]["work"] == (HQ + 2 * HK) * DIM and recs[1]["work"] == 4.0 * HQ * DIM


def test_main_runs(capsys):
    from sub_byte_mixed_amd import attn
    attn.main(["--workload", "tinyllama1b", "--reps", "1", "--length", "100"])
    assert capsys.readouterr().out.count("us") >= 4
