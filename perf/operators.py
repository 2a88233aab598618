"""The operators around the quantized linear layers, as cases to measure: RMS norm with the residual's
addition (forward with an FP8 output, backward), SwiGLU (forward with an FP8 output, backward) and the
product of one to sixteen tokens with block-scaled weights.

`own` False: run() computes them in elementary torch operations, in 32 bits; True: run() makes the calls
of sub_byte_mixed_amd. Sizes are those of the workloads in synth/ (hidden 2048, 4096 and 8192; FFN 5632,
11008 and 28672; 4096 and 8192 tokens, K/V projections of 256 outputs) and ragged ones next to them.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# Weight formats: id of the library, elements per scale (0: none), kind of the scale, tensor exponent.
FORMATS = {
    "fp8": (1, 0, "", True),
    "nvfp4": (2, 16, "e4m3", True),
    "mxfp4": (3, 32, "e8m0", False),
    "e4m3_b32": (4, 32, "e4m3", True),
    "e8m0_b16": (5, 16, "e8m0", False),
    "bf16_b16": (6, 16, "bf16", False),
    "bf16_b32": (7, 32, "bf16", False),
}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # the norm in front of a block's linears for one new token: latency of one small launch
        {"name": "norm_fwd_token", "op": "norm_fwd", "rows": 1, "cols": 2048, "x": "f32", "res": "bf16",
         "y": True, "fp8": False, "train": False},
        # a training step of the 1B block: Down's fp32 output joins the bf16 residual stream; bf16 for the
        # saved operand, FP8 codes for the next GEMM, the maximum for the next step's scale
        {"name": "norm_fwd_train", "op": "norm_fwd", "rows": 4096, "cols": 2048, "x": "f32", "res": "bf16",
         "y": True, "fp8": True, "train": True},
        # prefill of the 70B block: bf16 stream, only FP8 codes leave
        {"name": "norm_fwd_wide", "op": "norm_fwd", "rows": 4096, "cols": 8192, "x": "bf16", "res": "bf16",
         "y": False, "fp8": True, "train": False},
        # the backward of the 1B training step: dgrad's fp32 output in, residual gradient added
        {"name": "norm_bwd_train", "op": "norm_bwd", "rows": 4096, "cols": 2048, "dy": "f32", "dres": "bf16"},
        # a ragged batch and a width that no tile divides
        {"name": "norm_bwd_ragged", "op": "norm_bwd", "rows": 1003, "cols": 4104, "dy": "bf16", "dres": "bf16"},
        # the gate for one new token of the 1B block, on the two halves of one Gate/Up product
        {"name": "swiglu_fwd_token", "op": "swiglu_fwd", "rows": 1, "cols": 5632, "x": "f32", "y": True,
         "fp8": False, "train": False},
        # the 7B block's training step: fp32 GEMM outputs in, FP8 codes for Down out
        {"name": "swiglu_fwd_train", "op": "swiglu_fwd", "rows": 8192, "cols": 11008, "x": "f32", "y": False,
         "fp8": True, "train": True},
        # the backward of the 1B training step
        {"name": "swiglu_bwd_train", "op": "swiglu_bwd", "rows": 4096, "cols": 5632, "x": "f32"},
        # the smallest projection (K or V of the 1B block) for one token
        {"name": "gemv_kv_token", "op": "gemv", "tokens": 1, "n": 256, "k": 2048, "fmt": "nvfp4"},
        # the largest (Gate or Up of the 70B block) for one token
        {"name": "gemv_gate70b_token", "op": "gemv", "tokens": 1, "n": 28672, "k": 8192, "fmt": "nvfp4"},
        # Down of the 7B block for a few drafted tokens, MX-FP4
        {"name": "gemv_down7b_draft", "op": "gemv", "tokens": 4, "n": 4096, "k": 11008, "fmt": "mxfp4"},
        # Gate of the 7B block for a small decode batch
        {"name": "gemv_gate7b_batch", "op": "gemv", "tokens": 16, "n": 11008, "k": 4096, "fmt": "nvfp4"},
    ]


def _size(rng, low, high, step):
    """A multiple of `step` between low and high, spread over its logarithm."""
    v = step * max(1, round(math.exp(rng.uniform(math.log(low), math.log(high))) / step))
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "swiglu_fwd", "swiglu_bwd", "gemv", "gemv"])
    if op == "gemv":
        fmt = rng.choice(sorted(FORMATS))
        return {"op": op, "tokens": rng.choice([1, 1, 2, 3, 4, 6, 8, 11, 16]), "n": _size(rng, 200, 28672, 1),
                "k": _size(rng, 512, 8192, 32), "fmt": fmt}
    rows = _size(rng, 1, 4096, 1)
    if op == "norm_bwd":
        return {"op": op, "rows": rows, "cols": _size(rng, 256, 8192, 8), "dy": rng.choice(["bf16", "f32"]),
                "dres": rng.choice(["bf16", "f32", ""])}
    if op == "swiglu_bwd":
        return {"op": op, "rows": rows, "cols": _size(rng, 512, 11008, 8), "x": rng.choice(["bf16", "f32"])}
    fp8 = rng.random() < 0.6
    case = {"op": op, "rows": rows, "cols": _size(rng, 256, 8192, 16 if fp8 else 8), "x": rng.choice(["bf16", "f32"]),
            "y": not fp8 or rng.random() < 0.5, "fp8": fp8, "train": rng.random() < 0.5}
    if op == "norm_fwd":
        case["res"] = rng.choice(["bf16", "f32", ""])
    return case


# ------------------------------------------------------------------ inputs

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _stream(g, rows, cols):
    """Values of a residual stream: normal, with a few channels that are some times larger."""
    channel = 1.0 + 7.0 * (torch.rand(cols, generator=g, device="cuda") < 0.01)
    return _randn(g, rows, cols) * channel


def _weights(g, n, k, fmt):
    """Weights of standard deviation 0.02 in `fmt`, as a checkpoint holds them: codes, scales, exponent."""
    _, block, kind, texp = FORMATS[fmt]
    w = 0.02 * _randn(g, n, k)
    if fmt == "fp8":
        e = math.ceil(math.log2(float(w.abs().amax()) / 448.0))
        return {"codes": (w * 2.0 ** -e).to(torch.float8_e4m3fn).view(torch.uint8), "scales": None,
                "texp": torch.tensor([e], dtype=torch.int32, device="cuda")}
    e = math.ceil(math.log2(float(w.abs().amax()) / 2688.0)) if texp else 0
    w = (w * 2.0 ** -e).view(n, k // block, block)
    s = w.abs().amax(2) / 6.0
    if kind == "e4m3":
        stored = s.to(torch.float8_e4m3fn)
        s, stored = stored.float(), stored.view(torch.uint8)
    elif kind == "e8m0":
        x = torch.floor(torch.log2(s * 6.0)) - 2.0
        s, stored = torch.exp2(x), (x + 127.0).to(torch.uint8)
    else:
        stored = s.to(torch.bfloat16)
        s, stored = stored.float(), stored.view(torch.uint8)
    w = w / s.unsqueeze(2)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    c = (torch.bucketize(w.abs(), edges) + 8 * (w < 0)).to(torch.uint8).view(n, k)
    return {"codes": c[:, 0::2] | (c[:, 1::2] << 4), "scales": stored,
            "texp": torch.tensor([e], dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], {"case": case}

    def empty(dtype, *shape):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op == "gemv":
        m, n, k = case["tokens"], case["n"], case["k"]
        s["x"] = _stream(g, m, k).to(torch.bfloat16)
        s["w"] = _weights(g, n, k, case["fmt"])
        s["out"] = empty(torch.float32, m, n)
        return s
    rows, cols = case["rows"], case["cols"]
    if op in ("norm_fwd", "norm_bwd"):
        s["gamma"] = (1.0 + 0.1 * _randn(g, cols)).to(torch.bfloat16)
    if op == "norm_fwd":
        s["x"] = (0.5 * _stream(g, rows, cols)).to(TYPES[case["x"]])
        s["res"] = _stream(g, rows, cols).to(TYPES[case["res"]]) if case["res"] else None
        s["h"] = empty(torch.bfloat16, rows, cols) if case["res"] else None
        s["rstd"] = empty(torch.float32, rows) if case["train"] else None
        s["amax"] = 30.0 + torch.rand(1, generator=g, device="cuda")
    elif op == "norm_bwd":
        h = _stream(g, rows, cols)
        s["h"] = h.to(torch.bfloat16)
        s["rstd"] = torch.rsqrt(h.square().mean(1) + EPS)
        s["dy"] = (1e-3 * _randn(g, rows, cols)).to(TYPES[case["dy"]])
        s["dres"] = (1e-3 * _randn(g, rows, cols)).to(TYPES[case["dres"]]) if case["dres"] else None
        s["dx"], s["dgamma"] = empty(torch.bfloat16, rows, cols), empty(torch.float32, cols)
    else:
        both = (1.5 * _stream(g, rows, 2 * cols)).to(TYPES[case["x"]])  # the two halves of one product's output
        s["gate"], s["up"] = both[:, :cols], both[:, cols:]
        s["amax"] = 400.0 + torch.rand(1, generator=g, device="cuda")
        if op == "swiglu_bwd":
            s["dy"] = (1e-3 * _randn(g, rows, cols)).to(TYPES[case["x"]])
            s["dgate"], s["dup"] = empty(torch.bfloat16, rows, cols), empty(torch.bfloat16, rows, cols)
    if op in ("norm_fwd", "swiglu_fwd"):
        s["y"] = empty(torch.bfloat16, rows, cols) if case["y"] else None
        s["codes"] = empty(torch.uint8, rows, cols) if case["fp8"] else None
        s["texp"] = torch.zeros(1, dtype=torch.int32, device="cuda") if case["fp8"] else None
        s["stats"] = torch.zeros(1, 3, dtype=torch.float64, device="cuda") if case["fp8"] and case["train"] else None
    return s


# ------------------------------------------------------------------ plain form

def _plain_out(s, y, more):
    """y in bf16 and in FP8 with the power-of-two scale of the supplied maximum, as the case asks."""
    case, out = s["case"], dict(more)
    if case["y"]:
        out["y"] = y.to(torch.bfloat16)
    if case["fp8"]:
        m, e = torch.frexp(s["amax"])
        e = (e - 9 + (m > 0.875)).to(torch.int32)  # smallest e with amax * 2^-e <= 448
        out["codes"] = torch.clamp(torch.ldexp(y, -e), -448.0, 448.0).to(torch.float8_e4m3fn)
        out["texp"] = e
        if case["train"]:
            out["amax"] = y.abs().amax().reshape(1)
    return out


def _plain_weights(w, fmt):
    _, block, kind, texp = FORMATS[fmt]
    codes = w["codes"]
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        nibbles = torch.stack((codes & 15, codes >> 4), dim=2).view(codes.shape[0], -1)
        v = torch.tensor(E2M1, device="cuda")[nibbles.int()]
        if kind == "e4m3":
            scale = w["scales"].view(torch.float8_e4m3fn).float()
        elif kind == "e8m0":
            scale = torch.exp2(w["scales"].float() - 127.0)
        else:
            scale = w["scales"].view(torch.bfloat16).float()
        v = (v.view(v.shape[0], -1, block) * scale.unsqueeze(2)).view(v.shape)
    return torch.ldexp(v, w["texp"]) if texp else v


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "gemv":
        return s["x"].float() @ _plain_weights(s["w"], case["fmt"]).t()
    if op == "norm_fwd":
        h = s["x"].float()
        if case["res"]:
            h = h + s["res"].float()
        r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        more = {"h": h.to(torch.bfloat16)} if case["res"] else {}
        if case["train"]:
            more["rstd"] = r.view(-1)
        return _plain_out(s, h * r * s["gamma"].float(), more)
    if op == "norm_bwd":
        dy = s["dy"].float()
        r = s["rstd"].unsqueeze(1)
        xh = s["h"].float() * r
        d = dy * s["gamma"].float()
        dx = r * (d - xh * (d * xh).mean(1, keepdim=True))
        if case["dres"]:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(torch.bfloat16), "dgamma": (dy * xh).sum(0)}
    g, u = s["gate"].float(), s["up"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    if op == "swiglu_fwd":
        return _plain_out(s, g * sig * u, {})
    dy = s["dy"].float()
    return {"dgate": (dy * u * sig * (1.0 + g * (1.0 - sig))).to(torch.bfloat16), "dup": (dy * g * sig).to(torch.bfloat16)}


# ------------------------------------------------------------------ the framework's calls

def _own_out(s, y, q, stats, more):
    case, out = s["case"], dict(more)
    if case["y"]:
        out["y"] = y
    if case["fp8"]:
        out["codes"] = q.codes.view(torch.float8_e4m3fn)
        out["texp"] = q.texp
        if case["train"]:
            out["amax"] = stats.view(torch.float32)[0, 4:5]
    return out


def _own(s):
    import sub_byte_mixed_amd as S
    case = s["case"]
    op = case["op"]
    if op == "gemv":
        w = s["w"]
        w = S.QuantizedTensor(FORMATS[case["fmt"]][0], case["n"], case["k"], s["x"].device, codes=w["codes"],
                              scales=w["scales"], texp=w["texp"])
        return S.qgemv(s["x"], w, y=s["out"])
    if op == "norm_bwd":
        dx, dgamma = S.rmsnorm_bwd(s["dy"], s["h"], s["gamma"], s["rstd"], dres=s["dres"], dx=s["dx"], dgamma=s["dgamma"])
        return {"dx": dx, "dgamma": dgamma}
    if op == "swiglu_bwd":
        dgate, dup = S.swiglu_bwd(s["dy"], s["gate"], s["up"], dgate=s["dgate"], dup=s["dup"])
        return {"dgate": dgate, "dup": dup}
    q = None
    if case["fp8"]:
        q = S.QuantizedTensor(S.FP8, case["rows"], case["cols"], s["codes"].device, codes=s["codes"], texp=s["texp"])
    if op == "norm_fwd":
        y, h, rstd, q, stats = S.rmsnorm_fwd(
            s["x"], s["gamma"], EPS, res=s["res"], h=s["h"], y=s["y"], rstd=s["rstd"], q=q, with_y=case["y"],
            with_rstd=case["train"], amax=s["amax"], stats=s["stats"], with_stats=case["train"])
        more = {"h": h} if case["res"] else {}
        if case["train"]:
            more["rstd"] = rstd
        return _own_out(s, y, q, stats, more)
    y, q, stats = S.swiglu_fwd(s["gate"], s["up"], y=s["y"], q=q, with_y=case["y"], amax=s["amax"], stats=s["stats"],
                               with_stats=case["train"])
    return _own_out(s, y, q, stats, {})


def run(s):
    return _own(s) if own else _plain(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "gemv":
        _, block, kind, texp = FORMATS[case["fmt"]]
        m, n, k = case["tokens"], case["n"], case["k"]
        weight = n * k if block == 0 else n * k // 2 + n * (k // block) * (2 if kind == "bf16" else 1)
        return {"bytes": weight + 2 * m * k + 4 * m * n, "flops": 2 * m * n * k}
    size = {"bf16": 2, "f32": 4, "": 0}
    rows, cols = case["rows"], case["cols"]
    e = rows * cols
    if op == "norm_bwd":
        return {"bytes": e * (size[case["dy"]] + 2 + size[case["dres"]] + 2) + 4 * rows + 6 * cols, "flops": 9 * e}
    if op == "swiglu_bwd":
        return {"bytes": e * (3 * size[case["x"]] + 4), "flops": 12 * e}
    out = (2 if case["y"] else 0) + (1 if case["fp8"] else 0)
    if op == "swiglu_fwd":
        return {"bytes": e * (2 * size[case["x"]] + out), "flops": 6 * e}
    return {"bytes": e * (size[case["x"]] + size[case["res"]] + (2 if case["res"] else 0) + out) + 2 * cols
            + (4 * rows if case["train"] else 0), "flops": 6 * e}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    """Each output's value before the rounding to its own type; the FP8 codes' in units of their scale."""
    s = prepare(case, seed)
    op = case["op"]

    def wide(name):
        return s[name].to(torch.float64)

    if op == "gemv":
        fmt, w = case["fmt"], s["w"]
        _, block, kind, texp = FORMATS[fmt]
        x = wide("x")
        parts = []
        for a in range(0, case["n"], 4096):  # rows at a time, to bound the memory
            codes = w["codes"][a:a + 4096]
            if fmt == "fp8":
                v = codes.view(torch.float8_e4m3fn).to(torch.float64)
            else:
                v = torch.empty(codes.shape[0], case["k"], dtype=torch.float64, device="cuda")
                for half in (0, 1):
                    c = (codes >> (4 * half)) & 15
                    mag = (c & 7).to(torch.float64)
                    low, high = 0.5 * mag, (2.0 + (c & 1)) * torch.exp2(((c & 7) >> 1).to(torch.float64) - 2.0)
                    v[:, half::2] = torch.where(mag < 2, low, high) * (1.0 - 2.0 * (c >> 3))
                sc = w["scales"][a:a + 4096]
                if kind == "e4m3":
                    sc = sc.view(torch.float8_e4m3fn).to(torch.float64)
                elif kind == "bf16":
                    sc = sc.view(torch.bfloat16).to(torch.float64)
                else:
                    sc = torch.exp2(sc.to(torch.float64) - 127.0)
                v = v * sc.repeat_interleave(block, dim=1)
            parts.append(x @ v.t().contiguous())
        y = torch.cat(parts, dim=1)
        return y * 2.0 ** int(w["texp"]) if texp else y
    if op == "norm_bwd":
        dy, h, gamma, r = wide("dy"), wide("h"), wide("gamma"), wide("rstd")
        n = h.shape[1]
        dot = (dy * gamma * h).sum(1) * r
        dx = r[:, None] * gamma * dy - (r * r * dot / n)[:, None] * h
        if case["dres"]:
            dx += wide("dres")
        return {"dx": dx, "dgamma": (dy * h * r[:, None]).sum(0)}
    if op in ("swiglu_fwd", "swiglu_bwd"):
        g, u = wide("gate"), wide("up")
        t = 0.5 * torch.tanh(0.5 * g)  # sigmoid(g) = 1/2 + t
        if op == "swiglu_bwd":
            dy = wide("dy")
            sig = 0.5 + t
            return {"dgate": dy * u * (sig + g * (0.25 - t * t)), "dup": dy * g * sig}
        y, out = g * torch.sigmoid(g) * u, {}
    else:
        h = wide("x") + wide("res") if case["res"] else wide("x")
        r = 1.0 / torch.sqrt((h * h).sum(1) / h.shape[1] + EPS)
        y, out = h * r[:, None] * wide("gamma"), {}
        if case["res"]:
            out["h"] = h
        if case["train"]:
            out["rstd"] = r
    if case["y"]:
        out["y"] = y
    if case["fp8"]:
        e = math.ceil(math.log2(float(s["amax"]) / 448.0))
        out["codes"] = torch.clamp(y * 2.0 ** -e, -448.0, 448.0)
        out["texp"] = torch.tensor([e], dtype=torch.int32, device="cuda")
        if case["train"]:
            out["amax"] = y.abs().amax().reshape(1)
    return out
