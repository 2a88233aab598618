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


def _mat(t: Optional[torch.Tensor], name: str, rows: int, cols: int, dev: int) -> Tuple:
    """(address, element type, leading dimension) of a matrix argument."""
    if t is None:
        return _ABSENT
    ty = _TYPES.get(t.dtype)
    shape = t.shape
    if ty is None or len(shape) != 2 or shape[0] != rows or shape[1] != cols or t.get_device() != dev:
        raise ValueError(f"{name} must be a bfloat16 or float32 tensor of shape ({rows}, {cols}) on GPU {dev}, got "
                         f"{t.dtype}, {tuple(shape)} on {t.device}")
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows == 1:                                            # one row: its stride says nothing
        ld = -(-cols // 8) * 8
    return t.data_ptr(), ty, ld


def _vec(t: Optional[torch.Tensor], name: str, n: int, dtypes, dev: int) -> Optional[int]:
    if t is None:
        return None
    if t.dtype not in dtypes or t.shape != (n,) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} in {' or '.join(map(str, dtypes))} on GPU {dev}, "
                         f"got {t.dtype}, {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _new(rows: int, cols: int, dtype, dev: int) -> torch.Tensor:
    """A matrix whose rows are 16-byte aligned (a view of padded rows where the width asks for it)."""
    pad = -(-cols // 8) * 8
    t = torch.empty((rows, pad), dtype=dtype, device=dev)
    return t if pad == cols else t[:, :cols]


# (codes, scales) of a quantized format in bytes, as multiples of 1/32 byte an element
_SIZES = {f: (16, 32 // blk * (2 if kind == "bf16" else 1)) for f, (blk, kind) in _S.FP4_LAYOUT.items()}
_SIZES.update({_S.FP8: (32, 0), _S.BF16: (64, 0)})


def _holds(t: Optional[torch.Tensor], size: int, dev: int) -> bool:
    return t is not None and t.get_device() == dev and t.nbytes >= size and t.is_contiguous()


def _operand(q: "_S.QuantizedTensor", name: str, dev: int):
    """Reference to a quantized operand's descriptor, once its buffers are known to hold it."""
    codes, scales = _SIZES.get(q.format, (64, 0))
    n = q.rows * q.k
    if not (_holds(q.codes, n * codes // 32, dev) and (not scales or _holds(q.scales, n * scales // 32, dev))
            and _holds(q.texp, 4, dev)):
        raise ValueError(f"{name}: codes, scales and texp must be contiguous on GPU {dev} and hold "
                         f"[{q.rows}][{q.k}] in format {q.format}")
    return ctypes.byref(q.desc())


def _scratch(ws: Optional[torch.Tensor], dev: int) -> Tuple[Optional[int], int]:
    """(address, bytes) of a workspace argument."""
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on GPU {dev}")
    return ws.data_ptr(), ws.nbytes


_current_device = getattr(torch._C, "_cuda_getDevice", None)             # absent from a build of torch without GPUs
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # handle of a device's current stream


def _device(t: torch.Tensor, fn) -> int:
    """Index of the GPU that the first argument of fn lies on."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"the first argument of {fn.__name__} must be a 2-D GPU tensor")
    return t.get_device()


def _elsewhere(fn, dev: int, stream, *args):
    """fn(*args) on device `dev` and on `stream` (a torch stream of that
    device, an object with a stream's handle as cuda_stream, a handle, or None
    for the device's current one): what it allocates then belongs to the stream
    that its kernels run on."""
    if stream is None:
        with torch.cuda.device(dev):
            return fn(*args)
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        stream = torch.cuda.ExternalStream(handle, dev) if handle else torch.cuda.default_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream= is a stream of GPU {stream.device_index}, the tensors of {fn.__name__} lie on GPU {dev}")
    with torch.cuda.stream(stream):
        return fn(*args)


_F32 = (torch.float32,)
_ANY = (torch.bfloat16, torch.float32)


def _quant_out(q, out_fmt, rows, cols, dev, amax, stats, with_stats, ws, sizer):
    """The quantized output of a forward call: (q, stats, ws, their arguments
    of the C call: descriptor, maximum, statistics, workspace address and
    size). The caller holds ws until that call has returned: memory given back
    before its kernels are enqueued may be another call's by then."""
    if q is None and out_fmt is None:
        if stats is not None:
            raise ValueError("stats belong to a quantized output (out_fmt or q)")
        return None, None, ws, (None, None, None, None, 0)
    if q is None:
        q = _S.QuantizedTensor(out_fmt, rows, cols, dev)
    elif out_fmt is not None and q.format != out_fmt:
        raise ValueError(f"q is in format {q.format}, out_fmt is {out_fmt}")
    if stats is None:
        stats = _S.new_stats(1, dev) if with_stats else None
    elif stats.get_device() != dev or stats.nbytes < _S.STATS_BYTES or not stats.is_contiguous():
        raise ValueError(f"stats must be a statistics tensor (new_stats) on GPU {dev}")
    pa = _S._amax_ptr(amax)
    if pa is not None and (amax.stats if isinstance(amax, _S.StatsAmax) else amax).get_device() != dev:
        raise ValueError(f"amax must lie on GPU {dev}")
    if ws is None and (stats is not None or (amax is None and q.format != _S.MXFP4)):
        ws = torch.empty(sizer(rows, cols, q.format), dtype=torch.uint8, device=dev)
    return q, stats, ws, (_operand(q, "q", dev), pa, _S._ptr(stats), *_scratch(ws, dev))


def rmsnorm_fwd(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5, res: Optional[torch.Tensor] = None,
                h: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                rstd: Optional[torch.Tensor] = None, q: Optional["_S.QuantizedTensor"] = None,
                with_y: bool = True, with_rstd: bool = True, h_dtype: torch.dtype = torch.bfloat16,
                y_dtype: torch.dtype = torch.bfloat16, out_fmt: Optional[int] = None, rounding: int = 0,
                seed: int = 0, tensor_id: int = 0, amax=None, stats: Optional[torch.Tensor] = None,
                with_stats: bool = True, ws: Optional[torch.Tensor] = None, stream=None):
    """snipop_rmsnorm_fwd: h = x + res, y = h / sqrt(mean h^2 + eps) * gamma.

    Returns (y, h, rstd, q, stats). h is the new residual stream (None where
    there is no res and no buffer for it; pass h=res or h=x to update in
    place, but not over an h that a rmsnorm_bwd has still to read), rstd what
    rmsnorm_bwd needs, q the quantized y (out_fmt FP8, NVFP4
    or MXFP4, or a QuantizedTensor to write into; None otherwise). amax: a
    supplied max|y| for its tensor scale, as in linear_fwd_save (unused without
    q)."""
    dev = _device(x, rmsnorm_fwd)
    if stream is not None or dev != _current_device():
        return _elsewhere(rmsnorm_fwd, dev, stream, x, gamma, eps, res, h, y, rstd, q, with_y, with_rstd, h_dtype, y_dtype,
                          out_fmt, rounding, seed, tensor_id, amax, stats, with_stats, ws)
    rows, cols = x.shape
    px = _mat(x, "x", rows, cols, dev)
    pr = _mat(res, "res", rows, cols, dev)
    pg = _vec(gamma, "gamma", cols, _ANY, dev)
    if h is None and res is not None:
        h = _new(rows, cols, h_dtype, dev)
    if y is None and with_y:
        y = _new(rows, cols, y_dtype, dev)
    if rstd is None and with_rstd:
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    L = _S.lib()
    q, stats, ws, (d, pa, ps, *pw) = _quant_out(q, out_fmt, rows, cols, dev, amax, stats, with_stats, ws,
                                                L.snipop_rmsnorm_fwd_workspace)
    _S._check(L.snipop_rmsnorm_fwd(
        *px, *pr, pg, _TYPES[gamma.dtype], rows, cols, eps, *_mat(h, "h", rows, cols, dev),
        *_mat(y, "y", rows, cols, dev), _vec(rstd, "rstd", rows, _F32, dev), d, rounding, seed, tensor_id, pa, ps, *pw,
        _current_stream(dev)))
    return y, h, rstd, q, stats


def rmsnorm_bwd(dy: torch.Tensor, h: torch.Tensor, gamma: torch.Tensor, rstd: torch.Tensor,
                dres: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                dgamma: Optional[torch.Tensor] = None, need_dx: bool = True, need_dgamma: bool = True,
                dx_dtype: torch.dtype = torch.bfloat16, ws: Optional[torch.Tensor] = None, stream=None):
    """snipop_rmsnorm_bwd: the gradients of y from rmsnorm_fwd. h: its h (x
    where there was no res); dres: the gradient that reaches h along the
    residual stream. Returns (dx, dgamma); dx is the gradient of x and of res."""
    dev = _device(dy, rmsnorm_bwd)
    if stream is not None or dev != _current_device():
        return _elsewhere(rmsnorm_bwd, dev, stream, dy, h, gamma, rstd, dres, dx, dgamma, need_dx, need_dgamma, dx_dtype,
                          ws)
    rows, cols = dy.shape
    py = _mat(dy, "dy", rows, cols, dev)
    ph = _mat(h, "h", rows, cols, dev)
    if dx is None and need_dx:
        dx = _new(rows, cols, dx_dtype, dev)
    if dgamma is None and need_dgamma:
        dgamma = torch.empty(cols, dtype=torch.float32, device=dev)
    L = _S.lib()
    if ws is None and dgamma is not None:
        ws = torch.empty(L.snipop_rmsnorm_bwd_workspace(rows, cols), dtype=torch.uint8, device=dev)
    _S._check(L.snipop_rmsnorm_bwd(
        *py, *ph, _vec(gamma, "gamma", cols, _ANY, dev), _TYPES[gamma.dtype], _vec(rstd, "rstd", rows, _F32, dev),
        *_mat(dres, "dres", rows, cols, dev), rows, cols, *_mat(dx, "dx", rows, cols, dev),
        _vec(dgamma, "dgamma", cols, _F32, dev), *_scratch(ws, dev), _current_stream(dev)))
    return dx, dgamma


def swiglu_fwd(gate: torch.Tensor, up: torch.Tensor, y: Optional[torch.Tensor] = None,
               q: Optional["_S.QuantizedTensor"] = None, with_y: bool = True,
               y_dtype: torch.dtype = torch.bfloat16, out_fmt: Optional[int] = None, rounding: int = 0,
               seed: int = 0, tensor_id: int = 0, amax=None, stats: Optional[torch.Tensor] = None,
               with_stats: bool = True, ws: Optional[torch.Tensor] = None, stream=None):
    """snipop_swiglu_fwd: y = gate * sigmoid(gate) * up. Returns (y, q,
    stats), with q, amax and stats as in rmsnorm_fwd. gate and up may be the
    two halves of one tensor's columns."""
    dev = _device(gate, swiglu_fwd)
    if stream is not None or dev != _current_device():
        return _elsewhere(swiglu_fwd, dev, stream, gate, up, y, q, with_y, y_dtype, out_fmt, rounding, seed, tensor_id, amax,
                          stats, with_stats, ws)
    rows, cols = gate.shape
    if up.dtype != gate.dtype:
        raise ValueError("gate and up must have the same type")
    pg, tg, lg = _mat(gate, "gate", rows, cols, dev)
    pu, _, lu = _mat(up, "up", rows, cols, dev)
    if y is None and with_y:
        y = _new(rows, cols, y_dtype, dev)
    L = _S.lib()
    q, stats, ws, (d, pa, ps, *pw) = _quant_out(q, out_fmt, rows, cols, dev, amax, stats, with_stats, ws,
                                                L.snipop_swiglu_fwd_workspace)
    _S._check(L.snipop_swiglu_fwd(
        pg, lg, pu, lu, tg, rows, cols, *_mat(y, "y", rows, cols, dev), d, rounding, seed, tensor_id, pa, ps, *pw,
        _current_stream(dev)))
    return y, q, stats


def swiglu_bwd(dy: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, dgate: Optional[torch.Tensor] = None,
               dup: Optional[torch.Tensor] = None, need_dgate: bool = True, need_dup: bool = True,
               dtype: torch.dtype = torch.bfloat16, stream=None):
    """snipop_swiglu_bwd: (dgate, dup) from the gradient of swiglu_fwd's y."""
    dev = _device(dy, swiglu_bwd)
    if stream is not None or dev != _current_device():
        return _elsewhere(swiglu_bwd, dev, stream, dy, gate, up, dgate, dup, need_dgate, need_dup, dtype)
    rows, cols = dy.shape
    if up.dtype != gate.dtype:
        raise ValueError("gate and up must have the same type")
    py = _mat(dy, "dy", rows, cols, dev)
    pg, tg, lg = _mat(gate, "gate", rows, cols, dev)
    pu, _, lu = _mat(up, "up", rows, cols, dev)
    if dgate is None and need_dgate:
        dgate = _new(rows, cols, dtype, dev)
    if dup is None and need_dup:
        dup = _new(rows, cols, dtype, dev)
    if dgate is not None and dup is not None and dgate.dtype != dup.dtype:
        raise ValueError("dgate and dup must have the same type")
    pdg, tdg, ldg = _mat(dgate, "dgate", rows, cols, dev)
    pdu, tdu, ldu = _mat(dup, "dup", rows, cols, dev)
    _S._check(_S.lib().snipop_swiglu_bwd(*py, pg, lg, pu, lu, tg, rows, cols, pdg, ldg, pdu, ldu, max(tdg, tdu),
                                         _current_stream(dev)))
    return dgate, dup


def qgemv(x: torch.Tensor, w: "_S.QuantizedTensor", y: Optional[torch.Tensor] = None,
          y_dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """snipop_qgemv: y [tokens, N] = x [tokens, K] . dequant(w)^T for 1 to 16
    tokens, x in bfloat16, w in any quantized format with K % 32 == 0."""
    dev = _device(x, qgemv)
    if stream is not None or dev != _current_device():
        return _elsewhere(qgemv, dev, stream, x, w, y, y_dtype)
    m, k = x.shape
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16")
    if k != w.k:
        raise ValueError(f"x has {k} columns, w K={w.k}")
    px, _, lx = _mat(x, "x", m, k, dev)
    n = w.rows
    if y is None:
        y = torch.empty((m, n), dtype=y_dtype, device=x.device)
    ty = _TYPES.get(y.dtype)
    if ty is None or y.shape != (m, n) or y.get_device() != dev or (n > 1 and y.stride(1) != 1):
        raise ValueError(f"y must be a bfloat16 or float32 tensor of shape ({m}, {n}) with unit column stride on "
                         f"{x.device}")
    ly = y.stride(0) if m > 1 else n
    _S._check(_S.lib().snipop_qgemv(px, lx, m, _operand(w, "w", dev), y.data_ptr(), ty, ly, _current_stream(dev)))
    return y
