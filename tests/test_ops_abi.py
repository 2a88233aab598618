"""include/snip_ops.h and its binding without a GPU: every declared function
is exported, workspaces are sized, and bad arguments are rejected with the
documented status before any HIP call (the device addresses below are made
up and never touched)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import sub_byte_mixed_amd as S
from sub_byte_mixed_amd import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x7F0000000000
BIG = 1 << 30


def at(i):
    return P + i * 0x1000000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(S.LIB_PATH):
        from sub_byte_mixed_amd import build
        build.build()
    return S.lib()


def header():
    return open(os.path.join(ROOT, "include", "snip_ops.h")).read()


def qdesc(fmt, rows, k, codes=at(8), scales=at(9), texp=at(10)):
    return S.QTensorDesc(fmt, 0, rows, k, codes, scales, texp)


def test_declared_functions_are_exported_and_bound(L):
    names = sorted(set(re.findall(r"\b(snipop_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", header(), flags=re.S))))
    out = subprocess.run(["nm", "-D", "--defined-only", S.LIB_PATH], capture_output=True, text=True).stdout
    assert names == sorted(set(re.findall(r"\bT (snipop_[a-z0-9_]+)", out)))
    assert names == sorted(ops.SIGS)


def test_constants_agree_with_the_header():
    value = {n: int(v) for n, v in re.findall(r"#define\s+(SNIPOP_\w+)\s+(\d+)", header())}
    assert value["SNIPOP_NORM_MAX_COLS"] == ops.NORM_MAX_COLS
    assert value["SNIPOP_QGEMV_MAX_TOKENS"] == ops.QGEMV_MAX_TOKENS
    assert value["SNIPOP_BF16"] == ops._TYPES[torch.bfloat16] and value["SNIPOP_F32"] == ops._TYPES[torch.float32]
    for kind in ("NORM", "GATE", "GEMV"):
        assert S.LAUNCH_KINDS[value[f"SNIPOP_LAUNCH_{kind}"]] == kind.lower()


def test_workspace_sizes(L):
    assert L.snipop_rmsnorm_fwd_workspace(4096, 2048, S.FP8) > 0
    assert L.snipop_rmsnorm_fwd_workspace(4096, 2048, S.BF16) == 0
    assert L.snipop_rmsnorm_fwd_workspace(4096, 2056, S.NVFP4) == 0          # cols % 16
    assert L.snipop_rmsnorm_fwd_workspace(4096, 2064, S.MXFP4) == 0          # cols % 32
    assert L.snipop_rmsnorm_fwd_workspace(0, 2048, S.FP8) == 0
    assert L.snipop_swiglu_fwd_workspace(1, 16, S.NVFP4) > 0
    assert L.snipop_swiglu_fwd_workspace(1, 16, S.MXFP4) == 0
    for rows in (1, 3, 4096, 1 << 33):
        for cols in (1, 7, 2048, ops.NORM_MAX_COLS):
            n = L.snipop_rmsnorm_bwd_workspace(rows, cols)
            assert 4 * cols <= n <= 4 * (cols + 8) * 1024 + 256
    assert L.snipop_rmsnorm_bwd_workspace(8, ops.NORM_MAX_COLS + 1) == 0


def norm_fwd(L, x=at(0), xt=0, ldx=64, res=at(1), rt=0, ldr=64, gamma=at(2), gt=0, rows=4, cols=64, eps=1e-5, h=at(3),
             ht=0, ldh=64, y=at(4), yt=0, ldy=64, rstd=at(5), out=None, rnd=0, amax=None, stats=None, ws=at(6), n=BIG):
    return L.snipop_rmsnorm_fwd(x, xt, ldx, res, rt, ldr, gamma, gt, rows, cols, eps, h, ht, ldh, y, yt, ldy, rstd,
                                None if out is None else ctypes.byref(out), rnd, 0, 0, amax, stats, ws, n, None)


def test_rmsnorm_fwd_validation(L):
    assert norm_fwd(L, x=None) == -1
    assert norm_fwd(L, gamma=None) == -1
    assert norm_fwd(L, h=None, y=None, rstd=None) == -1
    assert norm_fwd(L, stats=at(7)) == -1                                    # statistics of nothing
    assert norm_fwd(L, rows=0) == -2 and norm_fwd(L, rows=-1) == -2
    assert norm_fwd(L, cols=0) == -2
    assert norm_fwd(L, cols=ops.NORM_MAX_COLS + 1, ldx=1 << 20) == -2
    assert norm_fwd(L, rows=1 << 50) == -2
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm_fwd(L, eps=eps) == -2
    assert norm_fwd(L, ldx=56) == -2                                         # ld < cols
    assert norm_fwd(L, ldr=68) == -2                                         # bf16: ld % 8
    assert norm_fwd(L, xt=1, ldx=66) == -2                                   # fp32: ld % 4
    assert norm_fwd(L, ldy=1 << 41) == -2
    for k in ("xt", "rt", "gt", "ht", "yt"):
        assert norm_fwd(L, **{k: 2}) == -4, k
    for k, v in (("x", at(0) + 8), ("res", at(1) + 2), ("gamma", at(2) + 4), ("h", at(3) + 8), ("y", at(4) + 1),
                 ("rstd", at(5) + 2)):
        assert norm_fwd(L, **{k: v}) == -3, k
    ok = qdesc(S.FP8, 4, 64)
    assert norm_fwd(L, out=qdesc(S.BF16, 4, 64)) == -4
    assert norm_fwd(L, out=qdesc(S.FP4_E8M0_B16, 4, 64)) == -4
    assert norm_fwd(L, out=qdesc(S.FP8, 4, 32)) == -2
    assert norm_fwd(L, out=qdesc(S.FP8, 8, 64)) == -2
    assert norm_fwd(L, out=qdesc(S.NVFP4, 4, 64, scales=None)) == -1
    assert norm_fwd(L, out=qdesc(S.FP8, 4, 64, texp=None)) == -1
    assert norm_fwd(L, out=qdesc(S.FP8, 4, 64, codes=at(8) + 8)) == -3
    assert norm_fwd(L, out=ok, rnd=2) == -4
    assert norm_fwd(L, out=ok, amax=at(7) + 2) == -3
    assert norm_fwd(L, out=ok, stats=at(7) + 4) == -3
    assert norm_fwd(L, out=ok, ws=None) == -5
    assert norm_fwd(L, out=ok, n=64) == -5
    assert "workspace" in L.snip_last_error().decode()


def test_rmsnorm_bwd_validation(L):
    def bwd(dy=at(0), yt=0, ldy=64, h=at(1), ht=0, ldh=64, gamma=at(2), gt=0, rstd=at(3), dres=at(4), rt=0, ldr=64,
            rows=4, cols=64, dx=at(5), xt=0, ldx=64, dgamma=at(6), ws=at(7), n=BIG):
        return L.snipop_rmsnorm_bwd(dy, yt, ldy, h, ht, ldh, gamma, gt, rstd, dres, rt, ldr, rows, cols, dx, xt, ldx,
                                    dgamma, ws, n, None)
    for k in ("dy", "h", "gamma", "rstd"):
        assert bwd(**{k: None}) == -1, k
    assert bwd(dx=None, dgamma=None) == -1
    assert bwd(rows=0) == -2 and bwd(cols=0) == -2
    assert bwd(cols=ops.NORM_MAX_COLS + 8) == -2
    for k in ("ldy", "ldh", "ldr", "ldx"):
        assert bwd(**{k: 60}) == -2, k
    for k in ("yt", "ht", "gt", "rt", "xt"):
        assert bwd(**{k: -1}) == -4, k
    for k, v in (("dy", at(0) + 8), ("h", at(1) + 4), ("gamma", at(2) + 2), ("rstd", at(3) + 1), ("dres", at(4) + 8),
                 ("dx", at(5) + 2), ("dgamma", at(6) + 2), ("ws", at(7) + 8)):
        assert bwd(**{k: v}) == -3, k
    assert bwd(n=4 * 64 - 1) == -5 and bwd(ws=None) == -5


def test_swiglu_validation(L):
    def fwd(g=at(0), ldg=64, u=at(1), ldu=64, t=0, rows=4, cols=64, y=at(2), yt=0, ldy=64, out=None, rnd=0, amax=None,
            stats=None, ws=at(6), n=BIG):
        return L.snipop_swiglu_fwd(g, ldg, u, ldu, t, rows, cols, y, yt, ldy,
                                   None if out is None else ctypes.byref(out), rnd, 0, 0, amax, stats, ws, n, None)
    assert fwd(g=None) == -1 and fwd(u=None) == -1 and fwd(y=None) == -1
    assert fwd(rows=0) == -2 and fwd(cols=-3) == -2
    assert fwd(ldg=60) == -2 and fwd(ldu=32) == -2 and fwd(ldy=70) == -2
    assert fwd(t=2) == -4 and fwd(yt=3) == -4
    assert fwd(u=at(1) + 8) == -3
    assert fwd(out=qdesc(S.MXFP4, 4, 48), cols=48) == -2
    assert fwd(out=qdesc(S.NVFP4, 4, 64), n=0) == -5

    def bwd(dy=at(0), yt=0, ldy=64, g=at(1), ldg=64, u=at(2), ldu=64, t=0, rows=4, cols=64, dg=at(3), lddg=64,
            du=at(4), lddu=64, dt=0):
        return L.snipop_swiglu_bwd(dy, yt, ldy, g, ldg, u, ldu, t, rows, cols, dg, lddg, du, lddu, dt, None)
    assert bwd(dy=None) == -1 and bwd(g=None) == -1 and bwd(u=None) == -1
    assert bwd(dg=None, du=None) == -1
    assert bwd(rows=0) == -2 and bwd(cols=0) == -2
    for k in ("ldy", "ldg", "ldu", "lddg", "lddu"):
        assert bwd(**{k: 56}) == -2, k
    for k in ("yt", "t", "dt"):
        assert bwd(**{k: 7}) == -4, k
    assert bwd(du=at(4) + 8) == -3


def test_qgemv_validation(L):
    def gemv(x=at(0), ldx=64, m=1, w=qdesc(S.NVFP4, 8, 64), y=at(1), yt=1, ldy=8):
        return L.snipop_qgemv(x, ldx, m, None if w is None else ctypes.byref(w), y, yt, ldy, None)
    assert gemv(x=None) == -1 and gemv(w=None) == -1 and gemv(y=None) == -1
    assert gemv(w=qdesc(S.NVFP4, 8, 64, scales=None)) == -1
    assert gemv(m=0) == -2 and gemv(m=ops.QGEMV_MAX_TOKENS + 1) == -2
    assert gemv(w=qdesc(S.NVFP4, 8, 48)) == -2                               # K % 32
    assert gemv(w=qdesc(S.FP8, 8, 48)) == -2
    assert gemv(w=qdesc(S.NVFP4, 0, 64)) == -2
    assert gemv(w=qdesc(S.NVFP4, (1 << 31) + 1, 64), ldy=1 << 33) == -2
    assert gemv(ldx=56) == -2 and gemv(ldx=68) == -2 and gemv(ldy=7) == -2
    assert gemv(w=qdesc(S.BF16, 8, 64)) == -4 and gemv(w=qdesc(8, 8, 64)) == -4
    assert gemv(yt=2) == -4
    assert gemv(x=at(0) + 8) == -3 and gemv(y=at(1) + 4) == -3
    assert gemv(w=qdesc(S.NVFP4, 8, 64, codes=at(8) + 8)) == -3


def test_binding_wants_gpu_matrices():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: S.rmsnorm_fwd(x, torch.ones(64)), lambda: S.rmsnorm_bwd(x, x, torch.ones(64), torch.ones(4)),
                 lambda: S.swiglu_fwd(x, x), lambda: S.swiglu_bwd(x, x, x), lambda: S.qgemv(x, None)):
        with pytest.raises(ValueError):
            call()


def test_workspace_is_wanted_for_the_maximum_and_the_statistics(L):
    """Without either a call goes past the workspace's check: here to the
    error of a launch without a GPU, or none at all."""
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    for fmt, amax, stats, wanted in ((S.FP8, None, None, True), (S.FP8, at(7), None, False), (S.NVFP4, at(7), at(9), True),
                                     (S.MXFP4, None, None, False), (S.MXFP4, None, at(9), True)):
        rc = norm_fwd(L, out=qdesc(fmt, 4, 64), amax=amax, stats=stats, ws=None, n=0)
        assert (rc == -5) == wanted, (fmt, amax, stats, rc)
