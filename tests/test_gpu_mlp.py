"""The MLP half of a block (sub_byte_mixed_amd/mlp.py): the operators and the
linear layers together, training and decode, against float64; and every
operator captured in a HIP graph.

FP8 everywhere, so that quantization noise stays small: half a step of E4M3
is 2^-4, rms below 3.6 %, of two operands 5.1 % of a product. The output sees
three products' noise (Gate, Up, Down): 8.8 %, bound 15 %. Stochastic rounding
is off by up to a step, rms below 5.1 %, 7.2 % of a product: the gradients see
the forward's 8.8 % and at most three such products', 15 %, bound 30 %."""
import pytest
import torch

import sub_byte_mixed_amd as S
from sub_byte_mixed_amd.mlp import GatedMLP
from ops_common import BF, F32, f64, rand, say

pytestmark = pytest.mark.gpu


def make(hidden=256, ffn=512, fmt=S.FP8):
    w = [(1.0 + 0.1 * rand((hidden,), F32, 1)).to(BF), rand((2 * ffn, hidden), BF, 2, 0.05), rand((hidden, ffn), BF, 3, 0.05)]
    return w, GatedMLP(*[t.cuda() for t in w], fmt=fmt)


def reference(w, x, res, eps=1e-5):
    gamma, wgu, wd, x, res = (torch.from_numpy(f64(t)).requires_grad_() for t in (*w, x, res))
    h = x + res
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + eps) * gamma
    g, u = (y @ wgu.t()).chunk(2, dim=1)
    return (gamma, wgu, wd, x), h, (g * torch.sigmoid(g) * u) @ wd.t()


def off(got, want):
    want = want.detach()
    return float((got.detach().cpu().double() - want).norm() / want.norm())


def test_training_step():
    w, mlp = make()
    T, hidden = 256, 256
    x, res, dout, dh = (rand((T, hidden), BF, 10 + i) for i in range(4))
    leaves, h, out = reference(w, x, res)
    ((out * torch.from_numpy(f64(dout))).sum() + (h * torch.from_numpy(f64(dh))).sum()).backward()
    say("mlp training step")
    got, stream, saved = mlp.forward(x.cuda(), res.cuda())
    grads = mlp.backward(dout.cuda(), dh.cuda(), saved)
    assert off(got, out) < 0.15 and off(stream, h) < 2.0 ** -8
    for name, g, leaf in zip(("dx", "dgamma", "dw_gate_up", "dw_down"), grads, (leaves[3], leaves[0], leaves[1], leaves[2])):
        assert off(g, leaf.grad) < 0.30, name
    again = mlp.backward(dout.cuda(), dh.cuda(), saved)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("m", [1, 3, 16])
@pytest.mark.parametrize("fmt", [S.FP8, S.NVFP4, S.MXFP4])
def test_decode_step(m, fmt):
    """Against float64 with the weights that the codes stand for; what is left
    are the bf16 roundings of y and a, 2^-8 each, of a long sum's terms."""
    from oracle import ops as OO
    w, mlp = make(fmt=fmt)
    mlp.quantize_weights()
    wq = [torch.from_numpy(OO.dequantize(fmt, q.codes.cpu().numpy(), None if q.scales is None else q.scales.cpu().numpy(),
                                         int(q.texp.cpu()), q.rows, q.k)) for q in (mlp.q_gate_up, mlp.q_down)]
    x, res = rand((m, 256), BF, 20), rand((m, 256), BF, 21)
    say("mlp decode", fmt, m)
    stream = res.cuda()
    out = mlp.decode(x.cuda(), stream)
    _, h, want = reference((w[0], *wq), x, res)
    assert off(out, want) < 2.0 ** -6 and off(stream, h) < 2.0 ** -8


def test_decode_equals_the_calls():
    _, mlp = make(fmt=S.MXFP4)
    mlp.quantize_weights()
    x, res = rand((2, 256), BF, 30).cuda(), rand((2, 256), BF, 31).cuda()
    y, h, _, _, _ = S.rmsnorm_fwd(x, mlp.gamma, mlp.eps, res=res)
    gu = S.qgemv(y, mlp.q_gate_up)
    want = S.qgemv(S.swiglu_fwd(gu[:, :512], gu[:, 512:])[0], mlp.q_down)
    assert torch.equal(mlp.decode(x, res), want) and torch.equal(res, h)


def test_graph_replays():
    """Every operator in one captured graph; each replay after eager work on
    the same buffers, against the eager result."""
    T, C, N = 130, 1056, 96
    x, res, dy = (rand((T, C), t, 40 + i).cuda() for i, t in enumerate((F32, BF, F32)))
    gamma = rand((C,), BF, 43).cuda()
    w, _ = S.quantize(rand((N, C), BF, 44, 0.05).cuda(), S.ROWWISE, S.NVFP4)
    b = {k: torch.empty(s, dtype=t, device="cuda") for k, s, t in (
        ("h", (T, C), BF), ("y", (T, C), BF), ("rstd", (T,), F32), ("dx", (T, C), BF), ("dgamma", (C,), F32),
        ("a", (T, C), BF), ("dg", (T, C), BF), ("du", (T, C), BF), ("o1", (1, N), F32), ("o16", (16, N), F32))}
    q = {k: S.QuantizedTensor(f, T, C, "cuda") for k, f in (("n", S.NVFP4), ("g", S.FP8))}
    st = [S.new_stats(1, "cuda") for _ in range(2)]
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")

    def step():
        S.rmsnorm_fwd(x, gamma, 1e-5, res=res, h=b["h"], y=b["y"], rstd=b["rstd"], q=q["n"], stats=st[0], ws=ws)
        S.rmsnorm_bwd(dy, b["h"], gamma, b["rstd"], dres=res, dx=b["dx"], dgamma=b["dgamma"], ws=ws)
        S.swiglu_fwd(x, dy, y=b["a"], q=q["g"], stats=st[1], ws=ws)
        S.swiglu_bwd(dy, x, dy, dgate=b["dg"], dup=b["du"])
        S.qgemv(b["y"][:1], w, y=b["o1"])
        S.qgemv(b["y"][:16], w, y=b["o16"])
    outs = [*b.values(), q["n"].codes, q["n"].scales, q["n"].texp, q["g"].codes, q["g"].texp, *st]
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        say("graph replay", i)
        for t in outs:
            t.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), c.view(torch.uint8)) for a, c in zip(outs, want)), i


def test_launches_are_timed():
    S.timing_start(64)
    x = rand((64, 512), BF, 50).cuda()
    w, _ = S.quantize(rand((32, 512), BF, 51).cuda(), S.ROWWISE, S.FP8, with_stats=False)
    S.timing_read()
    S.timing_start(64)
    y, _, r, _, _ = S.rmsnorm_fwd(x, torch.ones(512, dtype=BF, device="cuda"), out_fmt=S.FP8)
    S.rmsnorm_bwd(y, x, torch.ones(512, dtype=BF, device="cuda"), r)
    S.swiglu_bwd(y, *([S.swiglu_fwd(x, y)[0]] * 2))
    S.qgemv(x[:2], w)
    recs, untimed = S.timing_read()
    assert [k["kind"] for k in recs] == ["amax", "norm", "finalize", "norm", "gate", "gate", "gemv"] and untimed == 0
    assert recs[-1]["work"] == 2.0 * 2 * 32 * 512 and all(k["ms"] > 0 for k in recs)
