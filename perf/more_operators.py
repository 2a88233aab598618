"""Attention over a paged cache held in 4 bits, as cases to measure: appending keys and values (with the
position rotation, read back as the values that are stored), and the attention of one to thousands of new
tokens a sequence over the cache.

`own` False: run() computes them in elementary torch operations, in 32 bits; True: run() makes the calls
of sub_byte_mixed_amd. Head layouts are those of the workloads in synth/ (hidden 2048 with K/V of 256: 32
heads of 64 over 4; hidden 4096: 32 heads of 128; hidden 8192 with K/V of 1024: 64 heads of 128 over 8),
token counts theirs (4096, 8192) and ragged ones next to them.

The cache, in pages of `page` tokens (a power of two from 16), E2M1 codes two to a byte, low nibble first:
  k_codes  [pages][kv_heads][page / 16][dim / 2 / p][16 tokens][p bytes]        p = 16 (8 where dim is 64)
  k_scales [pages][kv_heads][page / 16][dim / block / s][16 tokens][s]          s = 2 p / block, at least 1
  v_codes  [pages][kv_heads][page / 4][dim / 2 / v][4 tokens][v bytes]          v = 4 (2 where dim is 64)
  v_scales [pages][kv_heads][page / 4][dim / block][4 tokens]
block and scale: 16 and E4M3 under one power of two for all keys and one for all values (nvfp4), 32 and
E8M0 (mxfp4). Sequence b has lens[b] tokens, the last of them new; token t lies in page table[b][t / page].
"""
import math

import torch

own = False

FORMATS = {"nvfp4": (2, 16), "mxfp4": (3, 32)}     # id of the library, elements per scale
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TEXP = (-6, -8)                                    # of keys and values in nvfp4, from a calibration
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _case(name, op, fmt, seqs, new, length, spread, heads, page, **more):
    q_heads, kv_heads, dim = heads
    return {"name": name, "op": op, "fmt": fmt, "seqs": seqs, "new": new, "len": length, "spread": spread, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, **more}


H1B, H7B, H70B = (32, 4, 64), (32, 32, 128), (64, 8, 128)


def listed():
    return [
        # one new token of the 1B block, out of the QKV product's fp32 output: latency
        _case("append_token", "append", "nvfp4", 1, 1, 700, 0.0, H1B, 64, x="f32", rot=64, inter=False),
        # a decode step of 64 sequences, 70B block
        _case("append_batch", "append", "nvfp4", 64, 1, 8192, 0.8, H70B, 64, x="f32", rot=128, inter=False),
        # the prompt of the 7B block's workload
        _case("append_prompt", "append", "nvfp4", 1, 8192, 8192, 0.0, H7B, 128, x="f32", rot=128, inter=False),
        # prompts of odd lengths, neighbouring pairs, half of a head rotated
        _case("append_ragged", "append", "mxfp4", 5, 701, 1403, 0.9, H70B, 16, x="bf16", rot=64, inter=True),
        # one new token after a short prompt, 1B block: latency
        _case("attn_token", "attn", "nvfp4", 1, 1, 700, 0.0, H1B, 64, window=0, lse=False),
        # one long document, 70B block: few rows, a long axis
        _case("attn_long", "attn", "nvfp4", 1, 1, 65536, 0.0, H70B, 64, window=0, lse=False),
        # a serving batch of ragged lengths, 70B block: the cache's bytes
        _case("attn_batch", "attn", "nvfp4", 64, 1, 8192, 0.8, H70B, 64, window=0, lse=False),
        # a serving batch without shared heads, 7B block
        _case("attn_batch_heads", "attn", "mxfp4", 16, 1, 4096, 0.5, H7B, 16, window=0, lse=True),
        # drafted tokens to be checked, within a sliding window
        _case("attn_draft", "attn", "nvfp4", 16, 4, 6001, 0.5, H70B, 32, window=4096, lse=False),
        # the 1B block's prompt of 4096 tokens: matrix work
        _case("attn_prompt", "attn", "nvfp4", 1, 4096, 4096, 0.0, H1B, 64, window=0, lse=False),
        # a prompt's second chunk, 7B block: 2048 tokens after 4096 in the cache
        _case("attn_chunk", "attn", "nvfp4", 1, 2048, 6144, 0.0, H7B, 128, window=0, lse=False),
        # prompts and single tokens in one batch, heads of 256
        _case("attn_ragged", "attn", "mxfp4", 6, 333, 2777, 0.95, (16, 4, 256), 32, window=1000, lse=True),
    ]


def _spread(rng, low, high):
    """Between low and high, spread over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    fmt = rng.choice(["nvfp4", "nvfp4", "mxfp4"])
    heads = rng.choice([H1B, H7B, H70B, (16, 4, 256), (28, 4, 128), (12, 12, 64), (20, 2, 128), (8, 1, 256), (48, 3, 64)])
    page = rng.choice([16, 32, 64, 128])
    if rng.random() < 0.35:
        seqs = rng.choice([1, 1, 2, 5, 16, 64, 130])
        new = 1 if rng.random() < 0.4 else _spread(rng, 2, max(3, 4096 // seqs))
        case = _case("", "append", fmt, seqs, new, new + _spread(rng, 1, 4096), rng.choice([0.0, 0.5, 0.95]), heads, page,
                     x=rng.choice(["bf16", "f32"]), rot=rng.choice([0, 64, heads[2], heads[2]]), inter=rng.random() < 0.3)
    elif rng.random() < 0.65:                      # a decode step: one or a few tokens a sequence
        seqs = _spread(rng, 1, 128)
        most = min(65536, 64 * 4900 * 1024 // (seqs * heads[1] * heads[2]))
        case = _case("", "attn", fmt, seqs, rng.choice([1, 1, 1, 2, 4, 7]), _spread(rng, 8, most), rng.choice([0.0, 0.5, 0.95]),
                     heads, page, window=rng.choice([0, 0, 0, 512, 3000]), lse=rng.random() < 0.3)
    else:                                          # prompts
        seqs = rng.choice([1, 1, 2, 4, 9])
        new = _spread(rng, 8, 1500 // seqs)
        case = _case("", "attn", fmt, seqs, new, new + _spread(rng, 1, 2048), rng.choice([0.0, 0.5, 0.95]), heads, page,
                     window=rng.choice([0, 0, 0, 512]), lse=rng.random() < 0.3)
    del case["name"]
    return case


def _sizes(case):
    """(tokens, new tokens) of each sequence: the first has the most, the others down to a share of it."""
    n, spread = case["seqs"], case["spread"]
    share = [1.0 - spread * ((b * 37) % n) / n for b in range(n)]
    new = [max(1, round(case["new"] * s)) for s in share]
    return [max(round(case["len"] * s), m) for s, m in zip(share, new)], new


# ------------------------------------------------------------------ inputs

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _channels(g, heads, dim):
    """Keys have a few channels that are some times larger than the others."""
    return 1.0 + 5.0 * (torch.rand(heads, 1, dim, generator=g, device="cuda") < 0.02)


def _edges():
    """|r| lies above as many of these as the index of its E2M1 magnitude, ties to the even one."""
    below = torch.nextafter(torch.tensor([0.75, 1.75, 3.5]), torch.tensor(0.0)).tolist()
    return torch.tensor([0.25, below[0], 1.25, below[1], 2.5, below[2], 5.0], device="cuda")


def _quantize(x, fmt, texp):
    """Codes (one a byte), stored scales and the scales' values of x [..., dim]; blocks along the last axis."""
    block = FORMATS[fmt][1]
    x = x.unflatten(-1, (-1, block))
    most = x.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        x = x * 2.0 ** -texp
        six = torch.full((), 6.0, device="cuda")   # a tensor: a division by a number is a product with its inverse
        stored = torch.clamp(most * 2.0 ** -texp / six, max=448.0).to(torch.float8_e4m3fn)
        scale = stored.float()
        r = x * torch.where(scale > 0.0, torch.ones_like(scale) / scale, torch.zeros_like(scale))
        stored = stored.view(torch.uint8)
    else:
        e = torch.where(most > 0.0, torch.clamp(torch.frexp(most)[1] - 3, min=-127), torch.full_like(most, -127, dtype=torch.int32))
        stored, scale = (e + 127).to(torch.uint8), torch.exp2(e.float())
        r = torch.where(most > 0.0, x / scale, torch.zeros_like(x) * x)
    codes = (torch.bucketize(r.abs(), _edges()) + 8 * torch.signbit(r)).to(torch.uint8)
    return codes.flatten(-2), stored.squeeze(-1), scale


def _values(codes, scale, fmt, texp):
    """What codes (one a byte) stand for, in 32 bits."""
    v = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device="cuda")[codes.int()]
    v = (v.unflatten(-1, (-1, FORMATS[fmt][1])) * scale).flatten(-2)
    return v * 2.0 ** texp if fmt == "nvfp4" else v


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _pieces(case):
    """Bytes of a piece of a key, of its scales, of a value."""
    p = 8 if case["dim"] == 64 else 16
    return p, max(1, 2 * p // FORMATS[case["fmt"]][1]), p // 4


def _fill(g, cache, case, channels):
    """Keys and values of earlier tokens into every page, some pages at a time."""
    fmt, page, dim, (p, s, v) = case["fmt"], case["page"], case["dim"], _pieces(case)
    pages, heads = cache["k_codes"].shape[:2]
    step = max(1, (1 << 26) // (heads * page * dim))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        codes, stored, _ = _quantize(_randn(g, n, heads, page // 16, 16, dim) * channels[:, None], fmt, TEXP[0])
        cache["k_codes"][a:a + n] = _pack(codes).unflatten(-1, (-1, p)).transpose(3, 4)
        cache["k_scales"][a:a + n] = stored.unflatten(-1, (-1, s)).transpose(3, 4)
        codes, stored, _ = _quantize(0.5 * _randn(g, n, heads, page // 4, 4, dim), fmt, TEXP[1])
        cache["v_codes"][a:a + n] = _pack(codes).unflatten(-1, (-1, v)).transpose(3, 4)
        cache["v_scales"][a:a + n] = stored.transpose(3, 4)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dim, heads, page, fmt = case["dim"], case["kv_heads"], case["page"], case["fmt"]
    block = FORMATS[fmt][1]
    lens, new = _sizes(case)
    each = [-(-n // page) for n in lens]
    pages = sum(each) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((case["seqs"], max(each)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(each):
        table[b, :n] = order[at:at + n]
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device="cuda")

    p, each_s, v = _pieces(case)
    cache = {"k_codes": zeros(pages, heads, page // 16, dim // 2 // p, 16, p),
             "k_scales": zeros(pages, heads, page // 16, dim // block // each_s, 16, each_s),
             "v_codes": zeros(pages, heads, page // 4, dim // 2 // v, 4, v), "v_scales": zeros(pages, heads, page // 4, dim // block, 4)}
    channels = _channels(g, heads, dim)
    s = {"case": case, "cache": cache, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "cu": None if case["new"] == 1 else torch.tensor(cu, dtype=torch.int32, device="cuda"),
         "texp": torch.tensor(TEXP, dtype=torch.int32, device="cuda")}
    if case["op"] == "attn":
        _fill(g, cache, case, channels)
        s["q"] = (1.3 * _randn(g, cu[-1], case["q_heads"] * dim)).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        return s
    width = (case["q_heads"] + 2 * heads) * dim    # one product's output: queries, keys, values
    qkv = _randn(g, cu[-1], width)
    a, b = case["q_heads"] * dim, (case["q_heads"] + heads) * dim
    qkv[:, a:b] *= channels.flatten()
    qkv[:, b:] *= 0.5
    qkv = qkv.to(TYPES[case["x"]])
    s["q"], s["k"], s["v"] = qkv[:, :a], qkv[:, a:b], qkv[:, b:]
    s["out"] = torch.empty(cu[-1], a, dtype=torch.bfloat16, device="cuda")
    s["cos"] = s["sin"] = None
    if case["rot"]:                                # angles of 64 bits: far positions lose them in 32
        f = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        angle = torch.arange(max(lens), dtype=torch.float64, device="cuda")[:, None] * f
        s["cos"], s["sin"] = torch.cos(angle).float(), torch.sin(angle).float()
    return s


# ------------------------------------------------------------------ plain form

def _rows(s):
    """Sequence and position of each new token."""
    lens = s["lens"].long()
    if s["cu"] is None:
        return torch.arange(lens.numel(), device="cuda"), lens - 1
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(lens.numel(), device="cuda"), new, output_size=s["q"].shape[0])
    return seq, torch.arange(s["q"].shape[0], device="cuda") - s["cu"][1:].long()[seq] + lens[seq]


def _rotate(x, s, pos):
    case = s["case"]
    x = x.float().unflatten(1, (-1, case["dim"]))
    if not case["rot"]:
        return x
    c, t = s["cos"][pos].unsqueeze(1), s["sin"][pos].unsqueeze(1)
    x, rest = x[..., :case["rot"]], x[..., case["rot"]:]
    if case["inter"]:
        a, b = x[..., 0::2], x[..., 1::2]
        x = torch.stack((a * c - b * t, b * c + a * t), dim=-1).flatten(-2)
    else:
        a, b = x.chunk(2, dim=-1)
        x = torch.cat((a * c - b * t, b * c + a * t), dim=-1)
    return torch.cat((x, rest), dim=-1)


def _plain_append(s):
    case, cache = s["case"], s["cache"]
    fmt, page, (p, each_s, each_v) = case["fmt"], case["page"], _pieces(case)
    seq, pos = _rows(s)
    at, row = s["table"][seq, pos // page].long(), pos % page
    out = {"q": _rotate(s["q"], s, pos).flatten(1).to(torch.bfloat16)}
    k, stored, scale = _quantize(_rotate(s["k"], s, pos), fmt, TEXP[0])
    cache["k_codes"][at, :, row // 16, :, row % 16] = _pack(k).unflatten(-1, (-1, p))
    cache["k_scales"][at, :, row // 16, :, row % 16] = stored.unflatten(-1, (-1, each_s))
    out["k"] = _values(k, scale, fmt, TEXP[0]).flatten(1).to(torch.bfloat16)
    v, stored, scale = _quantize(s["v"].float().unflatten(1, (-1, case["dim"])), fmt, TEXP[1])
    cache["v_codes"][at, :, row // 4, :, row % 4] = _pack(v).unflatten(-1, (-1, each_v))
    cache["v_scales"][at, :, row // 4, :, row % 4] = stored
    out["v"] = _values(v, scale, fmt, TEXP[1]).flatten(1).to(torch.bfloat16)
    return out


def _read(codes, scales, s, which):
    """Cached values [sequence, kv head, token, dim], of what lies in [sequence, page, kv head, group of
    tokens, piece, token, byte]."""
    fmt = s["case"]["fmt"]
    codes, scales = (t.transpose(4, 5).flatten(5).flatten(3, 4) for t in (codes, scales))
    codes = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    scale = scales.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else torch.exp2(scales.float() - 127.0)
    return _values(codes, scale.unsqueeze(-1), fmt, TEXP[which]).transpose(1, 2).flatten(2, 3)


def _plain_attn(s):
    case, cache = s["case"], s["cache"]
    dim, heads, group = case["dim"], case["kv_heads"], case["q_heads"] // case["kv_heads"]
    table = s["table"].long().clamp(min=0)
    k = _read(cache["k_codes"][table], cache["k_scales"][table], s, 0)
    v = _read(cache["v_codes"][table], cache["v_scales"][table].unsqueeze(-1), s, 1)
    seq, pos = _rows(s)
    first = torch.zeros_like(s["lens"]) if s["cu"] is None else s["cu"][:-1]
    row = torch.zeros_like(seq) if s["cu"] is None else torch.arange(seq.numel(), device="cuda") - first[seq]
    q = torch.zeros(case["seqs"], case["new"], heads, group, dim, device="cuda")
    q[seq, row] = s["q"].float().unflatten(1, (heads, group, dim))
    at = torch.full((case["seqs"], case["new"]), -1, device="cuda")
    at[seq, row] = pos
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)     # [sequence, kv head, group x row, dim]
    x = torch.matmul(q, k.transpose(2, 3)).unflatten(2, (group, -1)) * (1.0 / math.sqrt(dim))
    key = torch.arange(k.shape[2], device="cuda")
    seen = key <= at[..., None]
    if case["window"]:
        seen &= key > at[..., None] - case["window"]
    x = torch.where(seen[:, None, None], x, torch.full((), -math.inf, device="cuda"))
    most = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - most)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul((p / total.clamp(min=1e-30)).flatten(2, 3), v).unflatten(2, (group, -1))
    out = {"out": o.permute(0, 3, 1, 2, 4)[seq, row].flatten(1).to(torch.bfloat16)}
    if case["lse"]:
        out["lse"] = (most + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2)[seq, row].flatten(1)
    return out


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    import sub_byte_mixed_amd as S
    case, c = s["case"], s["cache"]
    cache = S.KVCache(FORMATS[case["fmt"]][0], c["k_codes"], c["k_scales"], c["v_codes"], c["v_scales"],
                      s["texp"] if case["fmt"] == "nvfp4" else None)
    batch = S.KVBatch(s["table"], s["lens"], s["cu"])
    if case["op"] == "append":
        q = S.kv_append(s["k"], s["v"], cache, batch, q=s["q"], cos=s["cos"], sin=s["sin"], interleaved=case["inter"], q_out=s["out"])
        k, v = S.kv_gather(cache, batch, s["q"].shape[0])
        return {"q": q, "k": k, "v": v}
    out, lse = S.kv_attn(s["q"], cache, batch, window=case["window"], out=s["out"], with_lse=case["lse"])
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def run(s):
    if own:
        return _own(s)
    return _plain_append(s) if s["case"]["op"] == "append" else _plain_attn(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    lens, new = _sizes(case)
    dim, hq, hk, tokens = case["dim"], case["q_heads"], case["kv_heads"], sum(new)
    cached = 2 * hk * (dim // 2 + dim // FORMATS[case["fmt"]][1])      # bytes of a token
    if case["op"] == "append":
        size = {"bf16": 2, "f32": 4}[case["x"]]
        moved = size * (hq + 2 * hk) * dim + 2 * hq * dim + 2 * cached + 4 * hk * dim + 4 * case["rot"]
        return {"bytes": tokens * moved, "flops": tokens * (3 * case["rot"] * (hq + hk) + 8 * 2 * hk * dim)}
    window, keys, read = case["window"], 0, 0
    for n, m in zip(lens, new):
        full = [min(p + 1, window) if window else p + 1 for p in range(n - m, n)]
        keys += sum(full)
        read += min(n, window + m - 1) if window else n
    return {"bytes": read * cached + 4 * tokens * hq * dim + (4 * tokens * hq if case["lse"] else 0), "flops": 4 * dim * hq * keys}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _nearest(x, values):
    """Index of the nearest of ascending `values`, ties to the even index."""
    hi = torch.searchsorted(values, x).clamp(1, values.numel() - 1)
    lo = hi - 1
    a, b = x - values[lo], values[hi] - x
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def _exact_block(x, fmt, texp):
    """x [n, dim] in 64 bits as the values that the format holds. Its definition rounds a sixth of the
    largest magnitude, the inverse of the scale and the scaled value to 32 bits: in bf16 inputs ties are common."""
    wide = dict(dtype=torch.float64, device="cuda")
    block = FORMATS[fmt][1]
    e2m1 = torch.tensor(MAGNITUDES, **wide)
    parts = []
    for p in x.split(1 << 17):
        p = p.reshape(-1, block)
        most = p.abs().max(1, keepdim=True).values
        if fmt == "nvfp4":
            e4m3 = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119], **wide)
            s = e4m3[_nearest((most * 2.0 ** -texp / 6.0).float().double(), e4m3)] * 2.0 ** texp
        else:
            s = torch.where(most > 0, torch.exp2((torch.floor(torch.log2(most)) - 2.0).clamp(min=-127.0)), torch.zeros_like(most))
        r = torch.where(s > 0, (p.abs() * (1.0 / s).float().double()).float().double(), torch.zeros_like(p)).contiguous()
        parts.append((torch.sign(p) * e2m1[_nearest(r, e2m1)] * s).reshape(-1, x.shape[1]))
    return torch.cat(parts)


def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _sizes(case)
    dim, hq, hk, fmt = case["dim"], case["q_heads"], case["kv_heads"], case["fmt"]
    wide = dict(dtype=torch.float64, device="cuda")
    if case["op"] == "append":
        pos = torch.cat([torch.arange(n - m, n, device="cuda") for n, m in zip(lens, new)])

        def turned(name, heads):
            x = s[name].to(torch.float64).reshape(-1, heads, dim).clone()
            if case["rot"]:
                half = case["rot"] // 2
                i = torch.arange(half, device="cuda")
                a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)
                z = torch.complex(x[..., a], x[..., b]) * torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]
                x[..., a], x[..., b] = z.real, z.imag
            return x
        return {"q": turned("q", hq).reshape(-1, hq * dim),
                "k": _exact_block(turned("k", hk).reshape(-1, dim), fmt, TEXP[0]).reshape(-1, hk * dim),
                "v": _exact_block(s["v"].to(torch.float64).reshape(-1, dim), fmt, TEXP[1]).reshape(-1, hk * dim)}
    block = FORMATS[fmt][1]
    c = s["cache"]
    pieces, sums, at = [], [], 0
    for b, (n, m) in enumerate(zip(lens, new)):    # a sequence at a time, its tokens in order
        use = s["table"][b, : -(-n // case["page"])].long()

        def decoded(codes, scales, texp):          # [kv head, token, dim / 2 bytes], [kv head, token, dim / block]
            v = torch.empty(hk, n, dim, **wide)
            for half in (0, 1):
                nib = (codes >> (4 * half)) & 15
                mag, e = (nib & 1).to(torch.float64), ((nib >> 1) & 3).to(torch.float64)
                m1 = torch.where(e == 0, 0.5 * mag, (1.0 + 0.5 * mag) * torch.exp2(e - 1.0))
                v[..., half::2] = torch.where(nib >= 8, -m1, m1)
            if fmt == "nvfp4":
                man, e = (scales & 7).to(torch.float64), ((scales >> 3) & 15).to(torch.float64)
                sc = torch.where(e == 0, man / 8.0 * 2.0 ** -6, (1.0 + man / 8.0) * torch.exp2(e - 7.0)) * 2.0 ** texp
            else:
                sc = torch.exp2(scales.to(torch.float64) - 127.0)
            return v * sc.repeat_interleave(block, dim=-1)
        kc = c["k_codes"][use].permute(1, 0, 2, 4, 3, 5).reshape(hk, -1, dim // 2)[:, :n]
        ks = c["k_scales"][use].permute(1, 0, 2, 4, 3, 5).reshape(hk, -1, dim // block)[:, :n]
        vc = c["v_codes"][use].permute(1, 0, 2, 4, 3, 5).reshape(hk, -1, dim // 2)[:, :n]
        vs = c["v_scales"][use].permute(1, 0, 2, 4, 3).reshape(hk, -1, dim // block)[:, :n]
        k, v = decoded(kc, ks, TEXP[0]), decoded(vc, vs, TEXP[1])
        q = s["q"][at:at + m].to(torch.float64).reshape(m, hk, -1, dim).transpose(0, 1)
        group = q.shape[2]
        o, z = torch.empty(m, hk, group, dim, **wide), torch.empty(m, hk, group, **wide)
        p, key = torch.arange(n - m, n, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
        hide = (key > p) | (key <= p - case["window"]) if case["window"] else key > p
        for h in range(hk):
            x = (q[h].reshape(-1, dim) @ k[h].t().contiguous()).reshape(m, group, n) / math.sqrt(dim)
            x = x.masked_fill(hide[:, None], -math.inf)
            z[:, h] = torch.logsumexp(x, dim=2)
            o[:, h] = (torch.exp(x - z[:, h, :, None]).reshape(-1, n) @ v[h]).reshape(m, group, dim)
        pieces.append(o.reshape(m, -1))
        sums.append(z.reshape(m, -1))
        at += m
    out = {"out": torch.cat(pieces)}
    if case["lse"]:
        out["lse"] = torch.cat(sums)
    return out
