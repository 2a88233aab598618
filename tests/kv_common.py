"""Helpers of the tests of the 4-bit key/value cache."""
import math

import numpy as np
import torch

import sub_byte_mixed_amd as S
from oracle import formats as F
from oracle import kv as OK
from oracle import quantize as OQ
from ops_common import U, f64

TEXP = (-3, -5)


def make_cache(fmt, pages, page, heads, dim, seed, device="cuda"):
    """A cache of random codes whose scales are all NaN: a page as it may come."""
    g = torch.Generator().manual_seed(seed)
    shapes = S.kv.cache_shapes(fmt, pages, page, heads, dim)
    bufs = [torch.randint(0, 256, s, generator=g, dtype=torch.uint8) for s in shapes]
    nan = 0x7F if fmt == S.NVFP4 else 0xFF
    for t in (bufs[1], bufs[3]):
        t.fill_(nan)
    texp = torch.tensor(TEXP, dtype=torch.int32, device=device) if fmt == S.NVFP4 else None
    return S.KVCache(fmt, *[t.to(device) for t in bufs], texp)


def tokens_view(t, keys):
    """[pages, heads, tokens, bytes of a token] of a cache buffer, its own memory."""
    return OK.token_major(t.cpu().numpy(), keys)


def scale_views(cache):
    """Scale bytes as [pages, heads, group, token, ...] views that can be written."""
    return cache.k_scales.transpose(3, 4), cache.v_scales.transpose(3, 4)


class Paged:
    """Sequences of `lens` tokens, the last new[b] of them this call's, in
    shuffled pages of a cache that is NaN wherever no token lies. unmapped: the
    (sequence, page index) pairs whose table entry names no page. capacity:
    tokens that the table has room for at least: above 1280 the steps of a call
    are shared among workgroups and joined by a second launch."""

    def __init__(self, fmt, dim, heads, page, lens, new, seed=0, unmapped=(), one_each=False, spare=3, capacity=0):
        self.fmt, self.dim, self.heads, self.page, self.lens, self.new = fmt, dim, heads, page, list(lens), list(new)
        g = torch.Generator().manual_seed(seed + 1)
        each = [max(0, -(-n // page)) for n in lens]
        pages = sum(each) + spare
        self.cache = make_cache(fmt, pages, page, heads, dim, seed)
        order = torch.randperm(pages, generator=g).tolist()
        wide = max(each + [1, -(-capacity // page)])
        table = np.full((len(lens), wide + 2), -1, np.int32)
        at = 0
        for b, n in enumerate(each):
            table[b, :n] = order[at:at + n]
            at += n
        kind = g.initial_seed()
        bad = (-1, pages, 2 ** 31 - 1, -2 ** 31)
        for i, (b, j) in enumerate(unmapped):
            table[b, j] = bad[(i + kind) % 4]
        self.table = table[:, :wide]
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.rows = int(self.cu[-1])
        dev = torch.from_numpy(table).cuda()
        self.batch = S.KVBatch(dev[:, :wide], torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                               None if one_each else torch.from_numpy(self.cu).cuda())
        # scales of the tokens that are there, over a wide range
        lo, hi = (0x18, 0x58) if fmt == S.NVFP4 else (118, 134)
        for t in scale_views(self.cache):
            per = t.shape[3]                           # tokens of a group
            for b, n in enumerate(self.lens):
                for j in range(0, max(n, 0), per):
                    p = int(self.table[b, j // page])
                    if 0 <= p < pages:
                        cnt = min(per, n - j)
                        dst = t[p, :, j % page // per, :cnt]
                        dst.copy_(torch.randint(lo, hi, dst.shape, generator=g, dtype=torch.uint8))

    def mapped(self, b):
        n = max(self.lens[b], 0)
        t = self.table[b][np.arange(n) // self.page] if n else np.zeros(0, np.int32)
        return (t >= 0) & (t < self.cache.pages)

    def positions(self, b):
        return self.lens[b] - self.new[b] + np.arange(self.new[b])

    def views(self):
        """The cache's bytes, token-major: k, k scales, v, v scales [pages, heads, tokens, ...]."""
        c = self.cache
        return [tokens_view(t, keys) for t, keys in ((c.k_codes, True), (c.k_scales, True), (c.v_codes, False), (c.v_scales, False))]

    def stored(self, b, views):
        """Of sequence b's tokens [heads, tokens, ...]; what is not mapped reads as zeros."""
        n, ok = max(self.lens[b], 0), self.mapped(b)
        at = np.arange(n)
        p = np.where(ok, self.table[b][at // self.page] if n else 0, 0)
        out = []
        for x in views:
            x = x[p, :, at % self.page].copy()
            x[~ok] = 0
            out.append(x.transpose(1, 0, 2))
        return out

    def values(self, b, views=None):
        k, ks, v, vs = self.stored(b, views or self.views())
        e = TEXP if self.fmt == S.NVFP4 else (0, 0)
        return OK.values(self.fmt, k, ks, e[0]), OK.values(self.fmt, v, vs, e[1])

    def attention(self, q, scale=None, window=0):
        """Reference, and tolerances of out and lse, for q [rows, heads x group x dim]."""
        dim, heads = self.dim, self.heads
        scale = 1.0 / math.sqrt(dim) if scale is None else scale
        q = f64(q).reshape(q.shape[0], heads, -1, dim)
        out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
        tol_o, tol_l = np.zeros(q.shape), np.zeros(q.shape[:3])
        views = self.views()
        for b in range(len(self.lens)):
            r = slice(self.cu[b], self.cu[b + 1])
            k, v = self.values(b, views)
            for h in range(heads):
                o, z, a, size, keys = OK.attention(q[r, h], k[h], v[h], self.positions(b), self.mapped(b), scale, window)
                out[r, h], lse[r, h] = o, z
                # what a score is off by: dim + 4 roundings of fp32 and, in NVFP4, the queries' 2^-25 of their largest
                off = (dim + 4) * U * size
                if self.fmt == S.NVFP4 and k.shape[1]:
                    qmax = np.abs(q[r, h]).max(axis=2)
                    off = off + 2.0 ** -25 * qmax * np.abs(k[h]).sum(axis=1).max() * scale
                # a term: its score, exp2 and the argument's rounding (|score| of 1 + log2 e times size); the sum
                # over the keys in fp32; its rounding before the product (fp16: 2^-11, two parts of bf16: 2^-17)
                rel = off + 2.0 ** -22 + 4 * U * 1.45 * size
                half = 2.0 ** -11 if self.fmt == S.NVFP4 else 2.0 ** -17
                sums = (keys + 64) * U
                tol_o[r, h] = a * (2 * rel + half + 2 * sums)[..., None] + 2.0 ** -8 * np.abs(o)
                # p below fp16's normal range is off by 2^-25, where the largest is 2^7 at least
                if self.fmt == S.NVFP4 and k.shape[1]:
                    tol_o[r, h] += 2.0 ** -32 * keys[..., None] * np.abs(v[h]).max()
                # and a term below 2^-126 of the largest is lost, as is a product or an output of that size
                if k.shape[1]:
                    tol_o[r, h] += 2.0 ** -126 * (1 + keys[..., None] * (1 + np.abs(v[h]).max()))
                tol_l[r, h] = rel + sums + 2.0 ** -21 + 4 * U * np.abs(np.where(np.isfinite(z), z, 0.0))
        n = q.shape[0]
        return out.reshape(n, -1), lse.reshape(n, -1), tol_o.reshape(n, -1), tol_l.reshape(n, -1)

    def check(self, q, out, lse=None, scale=None, window=0, what=""):
        o, z, to, tl = self.attention(q, scale, window)
        n = self.rows
        g = f64(out)[:n]
        bad = ~(np.abs(g - o[:n]) <= to[:n])
        assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), g[bad][:4], o[:n][bad][:4], to[:n][bad][:4])
        if lse is not None:
            g, z = f64(lse)[:n], z[:n]
            bad = ~((np.abs(g - np.where(np.isfinite(z), z, 0.0)) <= tl[:n]) | ((g == z) & ~np.isfinite(z)))
            assert not bad.any(), (what, "lse", np.argwhere(bad)[:4].tolist(), g[bad][:4], z[bad][:4], tl[:n][bad][:4])


def peak(P, at):
    """Keys of zero, but ones for token `at` of sequence 0; values of one, but zeros for that token (times 2^TEXP)."""
    c, p, j = P.cache, int(P.table[0, at // P.page]), at % P.page
    one = 0x38 if P.fmt == S.NVFP4 else 127
    c.k_codes.zero_()
    c.v_codes.fill_(0x22)
    for t in (c.k_scales, c.v_scales):
        t.fill_(one)
    c.k_codes[p, :, j // 16, :, j % 16] = 0x22
    c.v_codes[p, :, j // 4, :, j % 4] = 0


def quantized(x, fmt, texp):
    """Codes [rows, dim / 2] and scales [rows, dim / block] of fp32 x [rows, dim]."""
    o = OQ.quantize(np.asarray(x, np.float32), fmt, "rne", 0, 0, amax=np.float32(2688.0 * 2.0 ** texp) if fmt == S.NVFP4 else None)
    return o["packed"], o["scales"]
