"""Attention over a key/value cache held in 4 bits (include/snip_kv.h).
Re-exported by the package:

  KVCache(fmt, ...), KVCache.empty(...)    -> the pages of a cache
  KVBatch(table, lens, cu)                 -> a call's sequences and their new tokens
  kv_append(k, v, cache, batch, q, ...)    -> rotated queries; keys and values go into the cache
  kv_attn(q, cache, batch, ...)            -> out, lse
  kv_gather(cache, batch, tokens, ...)     -> cached keys and values in bfloat16

As in the package, this module only marshals arguments: every step runs in the
HIP kernels of libsnip. Queries, keys and values are 2-D GPU tensors with a row
for each new token and heads * head_dim columns of unit stride; their row stride
must keep rows 16-byte aligned. Outputs are allocated where no buffer is passed.
Every call takes stream= (default: the current one of the tensors' device).
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple

import torch

import sub_byte_mixed_amd as _S
from . import ops as _ops
from .ops import _TYPES, _elsewhere, _scratch, _vec

_c = ctypes
_vp, _i, _l, _f, _sz = _c.c_void_p, _c.c_int, _c.c_int64, _c.c_float, _c.c_size_t


class CacheDesc(_c.Structure):
    """snipkv_cache."""
    _fields_ = [("format", _c.c_int32), ("page_size", _c.c_int32), ("kv_heads", _c.c_int32), ("head_dim", _c.c_int32),
                ("pages", _l), ("k_codes", _vp), ("k_scales", _vp), ("v_codes", _vp), ("v_scales", _vp), ("texp", _vp)]


class BatchDesc(_c.Structure):
    """snipkv_batch."""
    _fields_ = [("table", _vp), ("table_ld", _l), ("max_pages", _l), ("lens", _vp), ("cu", _vp), ("seqs", _l)]


_C, _B = _c.POINTER(CacheDesc), _c.POINTER(BatchDesc)
SIGS = {
    "snipkv_append": (_i, [_vp, _l, _l, _vp, _l, _vp, _l, _i, _l, _vp, _vp, _l, _l, _i, _vp, _C, _B, _vp, _l, _vp]),
    "snipkv_gather": (_i, [_C, _B, _l, _vp, _l, _vp, _l, _vp]),
    "snipkv_attn": (_i, [_vp, _l, _l, _l, _C, _B, _f, _l, _vp, _l, _vp, _vp, _sz, _vp]),
    "snipkv_attn_workspace": (_sz, [_l, _l, _l, _l, _l]),
}

MAX_PAGE_SIZE = 4096           # SNIPKV_MAX_PAGE_SIZE
HEAD_DIMS = (64, 128, 256)


_U8, _I32, _BF, _F32 = torch.uint8, torch.int32, torch.bfloat16, torch.float32


@functools.lru_cache(maxsize=256)
def cache_shapes(fmt: int, pages: int, page_size: int, kv_heads: int, head_dim: int) -> Tuple[tuple, ...]:
    """Shapes of k_codes, k_scales, v_codes and v_scales."""
    if fmt not in (_S.NVFP4, _S.MXFP4):
        raise ValueError(f"a cache is in format NVFP4 or MXFP4, got {fmt}")
    if head_dim not in HEAD_DIMS or page_size < 16 or page_size > MAX_PAGE_SIZE or page_size & (page_size - 1):
        raise ValueError(f"head_dim must be one of {HEAD_DIMS} and page_size a power of two in 16 .. {MAX_PAGE_SIZE}, "
                         f"got {head_dim} and {page_size}")
    block = _S.FP4_LAYOUT[fmt][0]
    p = 8 if head_dim == 64 else 16
    v, s = p // 4, max(1, 2 * p // block)
    return ((pages, kv_heads, page_size // 16, head_dim // 2 // p, 16, p),
            (pages, kv_heads, page_size // 16, head_dim // block // s, 16, s),
            (pages, kv_heads, page_size // 4, head_dim // 2 // v, 4, v),
            (pages, kv_heads, page_size // 4, head_dim // block, 4))


def _buffer(t: torch.Tensor, name: str, shape: tuple, dev: int) -> int:
    """Its address."""
    if t.dtype is _U8 and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous uint8 tensor of shape {shape} on GPU {dev}, got {t.dtype}, "
                     f"{tuple(t.shape)} on {t.device}")


def _kept(name: str) -> property:
    """A tensor whose address the library was given: it is written into in place
    (`t += 1` ends by assigning the same tensor), not replaced."""
    at = "_" + name

    def get(self):
        return getattr(self, at)

    def put(self, value):
        if value is not getattr(self, at):
            raise AttributeError(f"{name} of a {type(self).__name__} is not replaced: write into it in place, or make another "
                                 f"{type(self).__name__}")
    return property(get, put)


class KVCache:
    """Caller-owned buffers of a paged cache, uint8 in the shapes of
    cache_shapes(); texp (NVFP4): int32 [2], the powers of two that keys and
    values are stored under (x = code * scale * 2^texp), chosen once by the
    caller: the smallest e with max|x| <= 2688 * 2^e. The
    buffers are not replaced by others."""
    k_codes, k_scales, v_codes, v_scales, texp = map(_kept, ("k_codes", "k_scales", "v_codes", "v_scales", "texp"))

    def __init__(self, fmt: int, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor,
                 v_scales: torch.Tensor, texp: Optional[torch.Tensor] = None):
        if k_codes.dim() != 6:
            raise ValueError("k_codes must have the six dimensions of cache_shapes()")
        pages, heads, groups, pieces, _, p = k_codes.shape
        page, dim, dev = 16 * groups, 2 * pieces * p, k_codes.get_device()
        sk, ssk, sv, ssv = cache_shapes(fmt, pages, page, heads, dim)
        at = (_buffer(k_codes, "k_codes", sk, dev), _buffer(k_scales, "k_scales", ssk, dev),
              _buffer(v_codes, "v_codes", sv, dev), _buffer(v_scales, "v_scales", ssv, dev))
        if texp is None and fmt == _S.NVFP4:
            raise ValueError("an NVFP4 cache needs texp")
        self.format, self.pages, self.kv_heads, self.page_size, self.head_dim, self.device = fmt, pages, heads, page, dim, dev
        self._k_codes, self._k_scales, self._v_codes, self._v_scales, self._texp = k_codes, k_scales, v_codes, v_scales, texp
        self._desc = CacheDesc(fmt, page, heads, dim, pages, *at, _vec(texp, "texp", 2, (_I32,), dev))
        self.ref = ctypes.byref(self._desc)

    @classmethod
    def empty(cls, fmt: int, pages: int, page_size: int, kv_heads: int, head_dim: int, device,
              texp: Tuple[int, int] = (0, 0)) -> "KVCache":
        """A cache of new buffers, zeroed."""
        bufs = [torch.zeros(s, dtype=torch.uint8, device=device) for s in cache_shapes(fmt, pages, page_size, kv_heads, head_dim)]
        return cls(fmt, *bufs, torch.tensor(texp, dtype=torch.int32, device=device) if fmt == _S.NVFP4 else None)


class KVBatch:
    """The sequences of a call: table int32 [seqs, max_pages] (pages of each
    sequence in order), lens int32 [seqs] (the call's new tokens included), cu
    int32 [seqs + 1] (rows cu[b] .. cu[b + 1] are sequence b's new tokens, its
    last; None: one each). A table entry outside 0 .. pages - 1 is a page that
    is not mapped. The kernels read all three when they run: a captured call
    follows what its buffers hold. They are written into in place, not
    replaced."""
    table, lens, cu = map(_kept, ("table", "lens", "cu"))

    def __init__(self, table: torch.Tensor, lens: torch.Tensor, cu: Optional[torch.Tensor] = None):
        dev = table.get_device()
        if table.dtype is not _I32 or table.dim() != 2:
            raise ValueError(f"table must be a 2-D int32 tensor, got {table.dtype}, {tuple(table.shape)}")
        (n, wide), (ld, unit) = table.shape, table.stride()
        if unit != 1 and wide > 1:
            raise ValueError("table must have unit column stride")
        self._table, self._lens, self._cu, self.seqs, self.device = table, lens, cu, n, dev
        self._desc = BatchDesc(table.data_ptr(), ld if n > 1 else wide, wide, _vec(lens, "lens", n, (_I32,), dev),
                               _vec(cu, "cu", n + 1, (_I32,), dev), n)
        self.ref = ctypes.byref(self._desc)


_CPU = -1                      # get_device() of a CPU tensor


def _place(cache: KVCache, batch: KVBatch, fn) -> int:
    """The GPU that a call's cache and sequences lie on."""
    dev = cache.device
    if batch.device != dev or dev == _CPU:
        raise ValueError(f"the cache and the batch of {fn.__name__} must lie on one GPU, got {dev} and {batch.device}")
    return dev


def _heads(t: torch.Tensor, name: str, dev: int, dim: int, dtype) -> Tuple[int, int, int, int]:
    """(address, leading dimension, tokens, heads) of a matrix of heads."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be a 2-D {dtype} tensor on GPU {dev}, got "
                         f"{(t.dtype, tuple(t.shape), t.device) if isinstance(t, torch.Tensor) else type(t)}")
    (rows, cols), (ld, unit) = t.shape, t.stride()
    if cols % dim or cols == 0:
        raise ValueError(f"{name} must have columns of heads of {dim}, got {cols}")
    if unit != 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), ld if rows > 1 else cols, rows, cols // dim      # one row: its stride says nothing


def _same(got: Tuple[int, int, int, int], name: str, tokens: int, heads: int) -> Tuple[int, int]:
    if got[2] != tokens or got[3] != heads:
        raise ValueError(f"{name} must have {tokens} rows of {heads} heads, got {got[2]} of {got[3]}")
    return got[:2]


def kv_append(k: Optional[torch.Tensor], v: Optional[torch.Tensor], cache: KVCache, batch: KVBatch,
              q: Optional[torch.Tensor] = None, cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None,
              interleaved: bool = False, pos: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
              stream=None) -> Optional[torch.Tensor]:
    """snipkv_append: rotates q and k by the angles of their tokens' positions
    (cos, sin: float32 [positions, rot_dim / 2]; rot_dim a multiple of 64, the
    rest of a head stays as it is; None: no rotation) and writes k and v into
    the cache. q, k and v have one type, bfloat16 or float32 (the parts of one
    product's columns, for instance); k and v may be None: queries alone. pos:
    int32 row of the angles for each token, instead of its position. Returns q
    rotated, in bfloat16 (None without q); q_out may be q itself."""
    dev = _place(cache, batch, kv_append)
    if stream is not None or dev != _ops._current_device():
        return _elsewhere(kv_append, dev, stream, k, v, cache, batch, q, cos, sin, interleaved, pos, q_out)
    dim, hk = cache.head_dim, cache.kv_heads
    first = q if k is None else k
    if first is None or (k is None) != (v is None):
        raise ValueError("k and v are given together, or q alone")
    dtype = getattr(first, "dtype", None)
    ty = _TYPES.get(dtype)
    if ty is None:
        raise ValueError(f"q, k and v must be bfloat16 or float32, got {dtype}")
    pk = lk = pv = lv = pq = lq = po = lo = pc = ps = pp = None
    angles = half = heads = 0
    if k is not None:
        got = _heads(k, "k", dev, dim, dtype)
        tokens = got[2]
        pk, lk = _same(got, "k", tokens, hk)
        pv, lv = _same(_heads(v, "v", dev, dim, dtype), "v", tokens, hk)
    if q is not None:
        pq, lq, rows, heads = _heads(q, "q", dev, dim, dtype)
        if k is None:
            tokens = rows
        elif rows != tokens:
            raise ValueError(f"q must have {tokens} rows, got {rows}")
        if q_out is None:
            q_out, lo = q.new_empty((tokens, heads * dim), dtype=_BF), heads * dim
            po = q_out.data_ptr()
        else:
            po, lo = _same(_heads(q_out, "q_out", dev, dim, _BF), "q_out", tokens, heads)
    elif q_out is not None:
        raise ValueError("q_out belongs to q")
    if cos is not None or sin is not None:
        if (cos is None or sin is None or cos.dim() != 2 or cos.shape != sin.shape or cos.dtype is not _F32
                or sin.dtype is not _F32 or cos.get_device() != dev or sin.get_device() != dev or not cos.is_contiguous()
                or not sin.is_contiguous()):
            raise ValueError(f"cos and sin must be contiguous float32 tensors of one shape [positions, rot_dim / 2] on GPU {dev}")
        (angles, half), pc, ps = cos.shape, cos.data_ptr(), sin.data_ptr()
    if pos is not None:
        pp = _vec(pos, "pos", tokens, (_I32,), dev)
    _S._check(_S.lib().snipkv_append(pq, lq or 0, heads, pk, lk or 0, pv, lv or 0, ty, tokens, pc, ps, angles, 2 * half,
                                     interleaved, pp, cache.ref, batch.ref, po, lo or 0, _ops._current_stream(dev)))
    return q_out


def kv_gather(cache: KVCache, batch: KVBatch, tokens: Optional[int] = None, k: Optional[torch.Tensor] = None,
              v: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """snipkv_gather: (keys, values) of the batch's tokens as they are cached,
    [tokens, kv_heads * head_dim] in bfloat16; zeros where a position is not
    mapped. tokens: rows of new outputs, cu[-1] at least (default: one a
    sequence)."""
    dev = _place(cache, batch, kv_gather)
    if stream is not None or dev != _ops._current_device():
        return _elsewhere(kv_gather, dev, stream, cache, batch, tokens, k, v)
    dim, hk = cache.head_dim, cache.kv_heads
    if tokens is None:
        tokens = k.shape[0] if k is not None else v.shape[0] if v is not None else batch.seqs
    lk = lv = hk * dim
    if k is None:
        k = cache.k_codes.new_empty((tokens, lk), dtype=_BF)
        pk = k.data_ptr()
    else:
        pk, lk = _same(_heads(k, "k", dev, dim, _BF), "k", tokens, hk)
    if v is None:
        v = cache.k_codes.new_empty((tokens, lv), dtype=_BF)
        pv = v.data_ptr()
    else:
        pv, lv = _same(_heads(v, "v", dev, dim, _BF), "v", tokens, hk)
    _S._check(_S.lib().snipkv_gather(cache.ref, batch.ref, tokens, pk, lk, pv, lv, _ops._current_stream(dev)))
    return k, v


@functools.lru_cache(maxsize=256)
def _workspace(tokens: int, seqs: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return _S.lib().snipkv_attn_workspace(tokens, seqs, q_heads, kv_heads, head_dim)


def kv_attn(q: torch.Tensor, cache: KVCache, batch: KVBatch, scale: Optional[float] = None, window: int = 0,
            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, with_lse: bool = False,
            ws: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """snipkv_attn: attention of the new tokens over the cache, which holds
    their keys and values already; causal, within the last `window` keys where
    window > 0. q bfloat16 (kv_append's); scale: default 1 / sqrt(head_dim).
    Returns (out bfloat16, lse): lse float32 [tokens, q_heads], the log of the
    softmax's sum, where with_lse or a buffer asks for it. A row that sees no
    key has out = 0 and lse = -inf."""
    dev = _place(cache, batch, kv_attn)
    if stream is not None or dev != _ops._current_device():
        return _elsewhere(kv_attn, dev, stream, q, cache, batch, scale, window, out, lse, with_lse, ws)
    dim, hk = cache.head_dim, cache.kv_heads
    pq, lq, tokens, heads = _heads(q, "q", dev, dim, _BF)
    if out is None:
        out, lo = q.new_empty((tokens, heads * dim)), heads * dim
        po = out.data_ptr()
    else:
        po, lo = _same(_heads(out, "out", dev, dim, _BF), "out", tokens, heads)
    pl = None
    if lse is None and with_lse:
        lse = q.new_empty((tokens, heads), dtype=_F32)
    if lse is not None:
        if lse.dtype is not _F32 or lse.shape != (tokens, heads) or lse.get_device() != dev or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 tensor of shape ({tokens}, {heads}) on GPU {dev}")
        pl = lse.data_ptr()
    if ws is None:
        nw = _workspace(tokens, batch.seqs, heads, hk, dim)
        ws = q.new_empty(nw, dtype=_U8)
        pw = ws.data_ptr()
    else:
        pw, nw = _scratch(ws, dev)
    _S._check(_S.lib().snipkv_attn(pq, lq, heads, tokens, cache.ref, batch.ref, 1.0 / math.sqrt(dim) if scale is None else scale,
                                   window, po, lo, pl, pw, nw, _ops._current_stream(dev)))
    return out, lse
