"""The operators around the quantized linear layers (include/snip_ops.h): RMS
norm with the residual's addition, SwiGLU, and the product of a few tokens
with block-scaled weights. Re-exported by the package:

  rmsnorm_fwd(x, gamma, eps, res, ...)     -> y, h, rstd, quantized y, stats
  rmsnorm_bwd(dy, h, gamma, rstd, ...)     -> dx, dgamma
  swiglu_fwd(gate, up, ...)                -> y, quantized y, stats
  swiglu_bwd(dy, gate, up, ...)            -> dgate, dup
  qgemv(x, w, ...)                         -> y

As in the package, this module only marshals arguments: every step runs in
the HIP kernels of libsnip. Matrices are 2-D GPU tensors in bfloat16 or
float32 with unit column stride; their row stride must keep rows 16-byte
aligned. Outputs are allocated where no buffer is passed. Every call takes
stream= (default: the current one of the tensors' device).
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

import sub_byte_mixed_amd as _S

_c = ctypes
_vp, _i, _l, _f, _u64, _u32, _sz = (_c.c_void_p, _c.c_int, _c.c_int64, _c.c_float, _c.c_uint64, _c.c_uint32,
                                    _c.c_size_t)
_Q = _c.POINTER(_S.QTensorDesc)
_TAIL = [_Q, _i, _u64, _u32, _vp, _vp, _vp, _sz, _vp]        # out .. stream of the forward calls
SIGS = {
    "snipop_rmsnorm_fwd": (_i, [_vp, _i, _l, _vp, _i, _l, _vp, _i, _l, _l, _f, _vp, _i, _l, _vp, _i, _l, _vp] + _TAIL),
    "snipop_rmsnorm_bwd": (_i, [_vp, _i, _l, _vp, _i, _l, _vp, _i, _vp, _vp, _i, _l, _l, _l, _vp, _i, _l, _vp, _vp,
                                _sz, _vp]),
    "snipop_swiglu_fwd": (_i, [_vp, _l, _vp, _l, _i, _l, _l, _vp, _i, _l] + _TAIL),
    "snipop_swiglu_bwd": (_i, [_vp, _i, _l, _vp, _l, _vp, _l, _i, _l, _l, _vp, _l, _vp, _l, _i, _vp]),
    "snipop_qgemv": (_i, [_vp, _l, _l, _Q, _vp, _i, _l, _vp]),
    "snipop_rmsnorm_fwd_workspace": (_sz, [_l, _l, _i]),
    "snipop_rmsnorm_bwd_workspace": (_sz, [_l, _l]),
    "snipop_swiglu_fwd_workspace": (_sz, [_l, _l, _i]),
}

NORM_MAX_COLS = 16384          # SNIPOP_NORM_MAX_COLS
QGEMV_MAX_TOKENS = 16          # SNIPOP_QGEMV_MAX_TOKENS
_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_ABSENT = (None, 0, 0)


def _mat(t: Optional[torch.Tensor], name: str, shape, device) -> Tuple:
    """(address, element type, leading dimension) of a matrix argument."""
    if t is None:
        return _ABSENT
    ty = _TYPES.get(t.dtype)
    if ty is None:
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    if t.dim() != 2 or t.shape != shape:
        raise ValueError(f"{name} must be of shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor on {device}, got one on {t.device}")
    rows, cols = shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    ld = t.stride(0) if rows > 1 else -(-cols // 8) * 8      # one row: its stride says nothing
    return t.data_ptr(), ty, ld


def _vec(t: Optional[torch.Tensor], name: str, n: int, dtypes, device) -> Optional[int]:
    if t is None:
        return None
    if t.dtype not in dtypes or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} in {' or '.join(map(str, dtypes))}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor on {device}")
    return t.data_ptr()


def _new(shape, dtype, device) -> torch.Tensor:
    """A matrix whose rows are 16-byte aligned (a view of padded rows where the width asks for it)."""
    rows, cols = shape
    pad = -(-cols // 8) * 8
    t = torch.empty((rows, pad), dtype=dtype, device=device)
    return t if pad == cols else t[:, :cols]


def _placed(fn):
    """Run fn on its first argument's device and on `stream` (a torch stream
    or a handle; default: the current one): what it allocates then belongs to
    the stream that its kernels run on."""
    @functools.wraps(fn)
    def call(first, *args, stream=None, **kw):
        if not isinstance(first, torch.Tensor) or first.dim() != 2 or not first.is_cuda:
            raise ValueError(f"the first argument of {fn.__name__} must be a 2-D GPU tensor")
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = (torch.cuda.ExternalStream(int(stream), device=first.device) if int(stream)
                          else torch.cuda.default_stream(first.device))
            with torch.cuda.stream(stream):
                return fn(first, *args, **kw)
        if first.device.index != torch.cuda.current_device():
            with torch.cuda.device(first.device):
                return fn(first, *args, **kw)
        return fn(first, *args, **kw)
    return call


_F32 = (torch.float32,)
_ANY = (torch.bfloat16, torch.float32)


def _quant_out(q, out_fmt, shape, device, amax, stats, with_stats, ws, sizer):
    """The quantized output's arguments of a forward call: descriptor, stats, workspace."""
    if q is None and out_fmt is None:
        if stats is not None:
            raise ValueError("stats belong to a quantized output (out_fmt or q)")
        return None, None, None
    if q is None:
        q = _S.QuantizedTensor(out_fmt, shape[0], shape[1], device)
    elif out_fmt is not None and q.format != out_fmt:
        raise ValueError(f"q is in format {q.format}, out_fmt is {out_fmt}")
    if stats is None and with_stats:
        stats = _S.new_stats(1, device)
    if ws is None:
        ws = _S._workspace(sizer(shape[0], shape[1], q.format), device)
    return q, stats, ws


@_placed
def rmsnorm_fwd(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5, res: Optional[torch.Tensor] = None,
                h: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                rstd: Optional[torch.Tensor] = None, q: Optional["_S.QuantizedTensor"] = None,
                with_y: bool = True, with_rstd: bool = True, h_dtype: torch.dtype = torch.bfloat16,
                y_dtype: torch.dtype = torch.bfloat16, out_fmt: Optional[int] = None, rounding: int = 0,
                seed: int = 0, tensor_id: int = 0, amax=None, stats: Optional[torch.Tensor] = None,
                with_stats: bool = True, ws: Optional[torch.Tensor] = None):
    """snipop_rmsnorm_fwd: h = x + res, y = h / sqrt(mean h^2 + eps) * gamma.

    Returns (y, h, rstd, q, stats). h is the new residual stream (None where
    there is no res and no buffer for it; pass h=res or h=x to update in
    place), rstd what rmsnorm_bwd needs, q the quantized y (out_fmt FP8, NVFP4
    or MXFP4, or a QuantizedTensor to write into; None otherwise). amax: a
    supplied max|y| for its tensor scale, as in linear_fwd_save (unused without
    q)."""
    shape, dev = x.shape, x.device
    rows, cols = shape
    px = _mat(x, "x", shape, dev)
    pr = _mat(res, "res", shape, dev)
    pg = _vec(gamma, "gamma", cols, _ANY, dev)
    if h is None and res is not None:
        h = _new(shape, h_dtype, dev)
    if y is None and with_y:
        y = _new(shape, y_dtype, dev)
    if rstd is None and with_rstd:
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    L = _S.lib()
    q, stats, ws = _quant_out(q, out_fmt, shape, dev, amax, stats, with_stats, ws, L.snipop_rmsnorm_fwd_workspace)
    d = None if q is None else ctypes.byref(q.desc())
    _S._check(L.snipop_rmsnorm_fwd(
        *px, *pr, pg, _TYPES[gamma.dtype], rows, cols, eps, *_mat(h, "h", shape, dev), *_mat(y, "y", shape, dev),
        _vec(rstd, "rstd", rows, _F32, dev), d, rounding, seed, tensor_id, _S._amax_ptr(amax), _S._ptr(stats),
        _S._ptr(ws), 0 if ws is None else ws.numel(), _S._stream(None)))
    return y, h, rstd, q, stats


@_placed
def rmsnorm_bwd(dy: torch.Tensor, h: torch.Tensor, gamma: torch.Tensor, rstd: torch.Tensor,
                dres: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                dgamma: Optional[torch.Tensor] = None, need_dx: bool = True, need_dgamma: bool = True,
                dx_dtype: torch.dtype = torch.bfloat16, ws: Optional[torch.Tensor] = None):
    """snipop_rmsnorm_bwd: the gradients of y from rmsnorm_fwd. h: its h (x
    where there was no res); dres: the gradient that reaches h along the
    residual stream. Returns (dx, dgamma); dx is the gradient of x and of res."""
    shape, dev = dy.shape, dy.device
    rows, cols = shape
    py = _mat(dy, "dy", shape, dev)
    ph = _mat(h, "h", shape, dev)
    if dx is None and need_dx:
        dx = _new(shape, dx_dtype, dev)
    if dgamma is None and need_dgamma:
        dgamma = torch.empty(cols, dtype=torch.float32, device=dev)
    L = _S.lib()
    if ws is None and dgamma is not None:
        ws = _S._workspace(L.snipop_rmsnorm_bwd_workspace(rows, cols), dev)
    _S._check(L.snipop_rmsnorm_bwd(
        *py, *ph, _vec(gamma, "gamma", cols, _ANY, dev), _TYPES[gamma.dtype], _vec(rstd, "rstd", rows, _F32, dev),
        *_mat(dres, "dres", shape, dev), rows, cols, *_mat(dx, "dx", shape, dev),
        _vec(dgamma, "dgamma", cols, _F32, dev), _S._ptr(ws), 0 if ws is None else ws.numel(), _S._stream(None)))
    return dx, dgamma


@_placed
def swiglu_fwd(gate: torch.Tensor, up: torch.Tensor, y: Optional[torch.Tensor] = None,
               q: Optional["_S.QuantizedTensor"] = None, with_y: bool = True,
               y_dtype: torch.dtype = torch.bfloat16, out_fmt: Optional[int] = None, rounding: int = 0,
               seed: int = 0, tensor_id: int = 0, amax=None, stats: Optional[torch.Tensor] = None,
               with_stats: bool = True, ws: Optional[torch.Tensor] = None):
    """snipop_swiglu_fwd: y = gate * sigmoid(gate) * up. Returns (y, q,
    stats), with q, amax and stats as in rmsnorm_fwd. gate and up may be the
    two halves of one tensor's columns."""
    shape, dev = gate.shape, gate.device
    rows, cols = shape
    if up.dtype != gate.dtype:
        raise ValueError("gate and up must have the same type")
    pg, tg, lg = _mat(gate, "gate", shape, dev)
    pu, _, lu = _mat(up, "up", shape, dev)
    if y is None and with_y:
        y = _new(shape, y_dtype, dev)
    L = _S.lib()
    q, stats, ws = _quant_out(q, out_fmt, shape, dev, amax, stats, with_stats, ws, L.snipop_swiglu_fwd_workspace)
    d = None if q is None else ctypes.byref(q.desc())
    _S._check(L.snipop_swiglu_fwd(
        pg, lg, pu, lu, tg, rows, cols, *_mat(y, "y", shape, dev), d, rounding, seed, tensor_id, _S._amax_ptr(amax),
        _S._ptr(stats), _S._ptr(ws), 0 if ws is None else ws.numel(), _S._stream(None)))
    return y, q, stats


@_placed
def swiglu_bwd(dy: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, dgate: Optional[torch.Tensor] = None,
               dup: Optional[torch.Tensor] = None, need_dgate: bool = True, need_dup: bool = True,
               dtype: torch.dtype = torch.bfloat16):
    """snipop_swiglu_bwd: (dgate, dup) from the gradient of swiglu_fwd's y."""
    shape, dev = dy.shape, dy.device
    rows, cols = shape
    if up.dtype != gate.dtype:
        raise ValueError("gate and up must have the same type")
    py = _mat(dy, "dy", shape, dev)
    pg, tg, lg = _mat(gate, "gate", shape, dev)
    pu, _, lu = _mat(up, "up", shape, dev)
    if dgate is None and need_dgate:
        dgate = _new(shape, dtype, dev)
    if dup is None and need_dup:
        dup = _new(shape, dtype, dev)
    if dgate is not None and dup is not None and dgate.dtype != dup.dtype:
        raise ValueError("dgate and dup must have the same type")
    pdg, tdg, ldg = _mat(dgate, "dgate", shape, dev)
    pdu, tdu, ldu = _mat(dup, "dup", shape, dev)
    _S._check(_S.lib().snipop_swiglu_bwd(*py, pg, lg, pu, lu, tg, rows, cols, pdg, ldg, pdu, ldu, max(tdg, tdu),
                                         _S._stream(None)))
    return dgate, dup


@_placed
def qgemv(x: torch.Tensor, w: "_S.QuantizedTensor", y: Optional[torch.Tensor] = None,
          y_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """snipop_qgemv: y [tokens, N] = x [tokens, K] . dequant(w)^T for 1 to 16
    tokens, x in bfloat16, w in any quantized format with K % 32 == 0."""
    shape, dev = x.shape, x.device
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16")
    if shape[1] != w.k:
        raise ValueError(f"x has {shape[1]} columns, w K={w.k}")
    if w.codes.device != dev:
        raise ValueError(f"w must be on {dev}, is on {w.codes.device}")
    px, _, lx = _mat(x, "x", shape, dev)
    out = torch.Size((shape[0], w.rows))
    if y is None:
        y = torch.empty(out, dtype=y_dtype, device=dev)
    ty = _TYPES.get(y.dtype)
    if ty is None or y.shape != out or y.device != dev or (w.rows > 1 and y.stride(1) != 1):
        raise ValueError(f"y must be a bfloat16 or float32 tensor of shape {tuple(out)} with unit column stride on {dev}")
    ly = y.stride(0) if shape[0] > 1 else max(y.stride(0), w.rows)
    _S._check(_S.lib().snipop_qgemv(px, lx, shape[0], ctypes.byref(w.desc()), y.data_ptr(), ty, ly,
                                    _S._stream(None)))
    return y
