"""The attention half of a Llama-like block for serving, out of the library's
calls: RMS norm with the residual's addition, Q, K and V as one product with
quantized weights, rotation and append to a 4-bit key/value cache, attention
over it, O -- for prompts, and for a decode step of a few tokens. With
mlp.GatedMLP it makes a block.

[SNIP, Fig. 4]: Q, K, V and O among the block's linear layers; between them
stand the operators of include/snip_ops.h and include/snip_kv.h.

  python -m sub_byte_mixed_amd.attn [--workload tinyllama1b] [--fmt nvfp4] [--reps 20]

times both on random weights of a workload's shapes.
"""
from __future__ import annotations

import argparse
import os
import sys
from typing import Tuple

import torch

import sub_byte_mixed_amd as S


def angles(positions: int, rot_dim: int, base: float = 10000.0, device="cuda") -> Tuple[torch.Tensor, torch.Tensor]:
    """(cos, sin) of position * base^(-2 i / rot_dim), float32 [positions,
    rot_dim / 2], the angles in 64 bits."""
    f = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * f
    return torch.cos(a).float(), torch.sin(a).float()


class CachedAttention:
    """w_qkv bf16 [(q_heads + 2 kv_heads) * head_dim, hidden] (Q's rows, then
    K's, then V's), w_o bf16 [hidden, q_heads * head_dim], gamma [hidden],
    quantized once in `fmt`; cos, sin as kv_append takes them. hidden and all
    widths are multiples of 128."""

    def __init__(self, gamma: torch.Tensor, w_qkv: torch.Tensor, w_o: torch.Tensor, kv_heads: int, head_dim: int,
                 cos: torch.Tensor, sin: torch.Tensor, fmt: int = S.NVFP4, eps: float = 1e-5):
        hidden, wide = w_o.shape
        self.a, self.b = wide, wide + kv_heads * head_dim          # columns where K and V begin
        if wide % head_dim or w_qkv.shape != (self.b + kv_heads * head_dim, hidden) or gamma.shape != (hidden,):
            raise ValueError(f"w_qkv must be [{self.b + kv_heads * head_dim}, {hidden}] and gamma [{hidden}] for w_o [{hidden}, {wide}] "
                             f"and {kv_heads} kv heads of {head_dim}")
        self.gamma, self.cos, self.sin, self.fmt, self.eps = gamma, cos, sin, fmt, eps
        self.kv_heads, self.head_dim = kv_heads, head_dim
        self.q_qkv, _ = S.quantize(w_qkv, S.ROWWISE, fmt, with_stats=False)
        self.q_o, _ = S.quantize(w_o, S.ROWWISE, fmt, with_stats=False)

    def _attend(self, qkv: torch.Tensor, cache: "S.KVCache", batch: "S.KVBatch", window: int, ws) -> torch.Tensor:
        # rows of no sequence are left as they were: zeros
        q = None if batch.cu is None else torch.zeros((qkv.shape[0], self.a), dtype=torch.bfloat16, device=qkv.device)
        q = S.kv_append(qkv[:, self.a:self.b], qkv[:, self.b:], cache, batch, q=qkv[:, :self.a], cos=self.cos, sin=self.sin, q_out=q)
        return S.kv_attn(q, cache, batch, window=window, out=q, ws=ws)[0]

    def prompt(self, x: torch.Tensor, res: torch.Tensor, cache: "S.KVCache", batch: "S.KVBatch", window: int = 0, ws=None):
        """x: what joins the residual stream res, both [T, hidden], T a multiple
        of 128; rows from batch.cu[-1] on are padding, whose output is zero. res
        becomes the new stream, the tokens' keys and values go into the cache;
        returns the output [T, hidden] in fp32."""
        y, _, _, _, _ = S.rmsnorm_fwd(x, self.gamma, self.eps, res=res, h=res, with_rstd=False)
        qy, _ = S.quantize(y, S.ROWWISE, self.fmt, with_stats=False)
        o = self._attend(S.qgemm(qy, self.q_qkv), cache, batch, window, ws)
        qo, _ = S.quantize(o, S.ROWWISE, self.fmt, with_stats=False)
        return S.qgemm(qo, self.q_o)

    def decode(self, x: torch.Tensor, res: torch.Tensor, cache: "S.KVCache", batch: "S.KVBatch", window: int = 0, ws=None):
        """1 to 16 tokens, one a sequence or as batch.cu says: res [m, hidden]
        becomes the new stream; returns the output [m, hidden] in fp32."""
        y, _, _, _, _ = S.rmsnorm_fwd(x, self.gamma, self.eps, res=res, h=res, with_rstd=False)
        return S.qgemv(self._attend(S.qgemv(y, self.q_qkv), cache, batch, window, ws), self.q_o)


GRAPH_STEPS = 16


def main(argv=None) -> None:
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    import synth
    from sub_byte_mixed_amd.mlp import _time
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--workload", default="tinyllama1b", choices=[w for w in synth.WORKLOAD_ORDER if len(synth.WORKLOADS[w].layers) == 7])
    ap.add_argument("--fmt", default="nvfp4", choices=[S.FORMAT_NAMES[f] for f in (S.NVFP4, S.MXFP4)])
    ap.add_argument("--length", type=int, default=4096, help="tokens of each sequence in decoding")
    ap.add_argument("--reps", type=int, default=20)
    args = ap.parse_args(argv)
    wl = synth.WORKLOADS[args.workload]
    fmt = {v: k for k, v in S.FORMAT_NAMES.items()}[args.fmt]
    T, hidden, wide, kv = wl.tokens, wl.layer("Q").d_in, wl.layer("Q").d_out, wl.layer("K").d_out
    dim = 64 if hidden <= 2048 else 128
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def randn(*shape, scale=1.0):
        return (scale * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)

    n = max(T, args.length)
    att = CachedAttention(1.0 + randn(hidden, scale=0.1), randn(wide + 2 * kv, hidden, scale=0.02), randn(hidden, wide, scale=0.02),
                          kv // dim, dim, *angles(n, dim), fmt)
    page, each = 64, -(-n // 64)
    cache = S.KVCache.empty(fmt, 16 * each, page, kv // dim, dim, "cuda", texp=(-6, -6))

    def int32(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    table = torch.randperm(16 * each, generator=g, device="cuda").int().view(16, each)
    x, res = randn(T, hidden), randn(T, hidden)
    batch = S.KVBatch(table[:1], int32(T), int32(0, T))
    print(f"{wl.name} attention, {args.fmt}: prompt of {T} tokens {_time(lambda: att.prompt(x, res, cache, batch), args.reps):.0f} us", flush=True)
    for b in range(16):                                           # every sequence's cache filled
        att.prompt(x, res.clone(), cache, S.KVBatch(table[b:b + 1], int32(T), int32(0, T)))
    for m in (1, 4, 16):
        xd, rd = x[:m].clone(), res[:m].clone()
        batch = S.KVBatch(table[:m], int32(*[args.length] * m))
        att.decode(xd, rd, cache, batch)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):                             # several steps, as a model's blocks would be
            for _ in range(GRAPH_STEPS):
                att.decode(xd, rd, cache, batch)
        print(f"{wl.name} attention, {args.fmt}: decode step of {m} sequences of {args.length} tokens "
              f"{_time(lambda: att.decode(xd, rd, cache, batch), args.reps):.1f} us, in a graph of {GRAPH_STEPS} "
              f"{_time(graph.replay, args.reps) / GRAPH_STEPS:.1f} us", flush=True)


if __name__ == "__main__":
    main()
