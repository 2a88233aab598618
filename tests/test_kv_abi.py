"""include/snip_kv.h and its binding without a GPU: every declared function is
exported, workspaces are sized, and bad arguments are rejected with the
documented status before any HIP call (the device addresses below are made up
and never touched)."""
import ctypes
import os
import re
import subprocess

import pytest

import sub_byte_mixed_amd as S
from sub_byte_mixed_amd import kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x7F0000000000
BIG = 1 << 40
NULL, SHAPE, ALIGN, FORMAT, WORKSPACE = -1, -2, -3, -4, -5


def at(i):
    return P + i * 0x1000000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(S.LIB_PATH):
        from sub_byte_mixed_amd import build
        build.build()
    return S.lib()


def header():
    return open(os.path.join(ROOT, "include", "snip_kv.h")).read()


def test_status_codes():
    text = open(os.path.join(ROOT, "include", "snip.h")).read()
    codes = {n: int(v) for n, v in re.findall(r"#define\s+SNIP_E_(\w+)\s+\(?(-\d+)\)?", text)}
    assert (codes["NULL"], codes["SHAPE"], codes["ALIGN"], codes["FORMAT"], codes["WORKSPACE"]) == (NULL, SHAPE, ALIGN, FORMAT, WORKSPACE)


def test_declared_functions_are_exported_and_bound(L):
    text = re.sub(r"/\*.*?\*/", "", header(), flags=re.S)
    names = sorted(set(re.findall(r"\b(snipkv_[a-z0-9_]+)\s*\(", text)))
    out = subprocess.run(["nm", "-D", "--defined-only", S.LIB_PATH], capture_output=True, text=True).stdout
    assert names == sorted(set(re.findall(r"\bT (snipkv_[a-z0-9_]+)", out))) == sorted(kv.SIGS)


def test_constants_agree_with_the_header():
    value = {n: int(v) for n, v in re.findall(r"#define\s+(SNIPKV_\w+)\s+(\d+)", header())}
    assert value["SNIPKV_MAX_PAGE_SIZE"] == kv.MAX_PAGE_SIZE
    for kind in ("APPEND", "ATTN", "JOIN"):
        assert S.LAUNCH_KINDS[value[f"SNIPKV_LAUNCH_{kind}"]] == "kv_" + kind.lower()


def test_descriptors_match_the_c_structs(tmp_path):
    src = tmp_path / "sizes.c"
    fields = {"snipkv_cache": [n for n, _ in kv.CacheDesc._fields_], "snipkv_batch": [n for n, _ in kv.BatchDesc._fields_]}
    lines = [f'printf("%zu\\n", sizeof({t}));' + "".join(f'printf("%zu\\n", offsetof({t}, {f}));' for f in fs) for t, fs in fields.items()]
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "snip_kv.h"\nint main(void){' + "".join(lines) + "return 0;}")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    want = []
    for d in (kv.CacheDesc, kv.BatchDesc):
        want += [ctypes.sizeof(d)] + [getattr(d, n).offset for n, _ in d._fields_]
    assert got == want


def cache(fmt=S.NVFP4, page=64, heads=4, dim=128, pages=10, kc=at(0), ks=at(1), vc=at(2), vs=at(3), texp=at(4)):
    return kv.CacheDesc(fmt, page, heads, dim, pages, kc, ks, vc, vs, texp)


def batch(table=at(5), ld=8, wide=8, lens=at(6), cu=at(7), seqs=3):
    return kv.BatchDesc(table, ld, wide, lens, cu, seqs)


def ref(d):
    return None if d is None else ctypes.byref(d)


def append(L, q=at(8), ldq=1024, heads=8, k=at(9), ldk=512, v=at(10), ldv=512, ty=0, tokens=5, cos=at(11), sin=at(12), angles=100,
           rot=128, inter=0, pos=None, c=None, b=None, out=at(13), ldo=1024):
    c, b = cache() if c is None else c, batch() if b is None else b
    return L.snipkv_append(q, ldq, heads, k, ldk, v, ldv, ty, tokens, cos, sin, angles, rot, inter, pos, ref(c or None), ref(b or None),
                           out, ldo, None)


def attn(L, q=at(8), ldq=1024, heads=8, tokens=5, c=None, b=None, scale=0.1, window=0, out=at(9), ldo=1024, lse=None, ws=at(10), n=BIG):
    c, b = cache() if c is None else c, batch() if b is None else b
    return L.snipkv_attn(q, ldq, heads, tokens, ref(c or None), ref(b or None), scale, window, out, ldo, lse, ws, n, None)


def gather(L, c=None, b=None, tokens=5, k=at(8), ldk=512, v=at(9), ldv=512):
    c, b = cache() if c is None else c, batch() if b is None else b
    return L.snipkv_gather(ref(c or None), ref(b or None), tokens, k, ldk, v, ldv, None)


BAD_CACHES = [(dict(fmt=S.FP8), FORMAT), (dict(fmt=S.BF16), FORMAT), (dict(fmt=4), FORMAT), (dict(page=8), SHAPE), (dict(page=48), SHAPE),
              (dict(page=8192), SHAPE), (dict(page=0), SHAPE), (dict(page=-64), SHAPE), (dict(heads=0), SHAPE), (dict(heads=1025), SHAPE),
              (dict(dim=96), SHAPE), (dict(dim=0), SHAPE), (dict(dim=512), SHAPE), (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE),
              (dict(kc=None), NULL), (dict(ks=None), NULL), (dict(vc=None), NULL), (dict(vs=None), NULL), (dict(texp=None), NULL),
              (dict(kc=at(0) + 8), ALIGN), (dict(ks=at(0) + 4), ALIGN), (dict(vc=at(0) + 1), ALIGN), (dict(vs=at(0) + 2), ALIGN),
              (dict(texp=at(0) + 2), ALIGN)]
BAD_BATCHES = [(dict(table=None), NULL), (dict(lens=None), NULL), (dict(cu=None), SHAPE), (dict(seqs=0), SHAPE), (dict(seqs=(1 << 20) + 1), SHAPE),
               (dict(wide=0), SHAPE), (dict(ld=7), SHAPE), (dict(wide=1 << 25, ld=1 << 25), SHAPE), (dict(table=at(0) + 2), ALIGN),
               (dict(lens=at(0) + 1), ALIGN), (dict(cu=at(0) + 3), ALIGN), (dict(ld=1 << 41), SHAPE)]


@pytest.mark.parametrize("call", [append, attn, gather])
def test_caches_and_batches(L, call):
    for more, code in BAD_CACHES:
        assert call(L, c=cache(**more)) == code, more
    for more, code in BAD_BATCHES:
        assert call(L, b=batch(**more)) == code, more
    assert call(L, c=False) == NULL and call(L, b=False) == NULL
    for tokens in (0, -1, (1 << 20) + 1):
        assert call(L, tokens=tokens) == SHAPE
    assert L.snip_last_error()


def test_append_validation(L):
    for more, code in [(dict(q=None, k=None, v=None, out=None), NULL), (dict(v=None), NULL), (dict(k=None), NULL), (dict(out=None), NULL),
                       (dict(q=None), NULL), (dict(ty=2), FORMAT), (dict(heads=6), SHAPE), (dict(heads=0), SHAPE), (dict(heads=1028), SHAPE),
                       (dict(ldq=1016), SHAPE), (dict(ldq=1028), SHAPE), (dict(ldk=504), SHAPE), (dict(ldv=516), SHAPE), (dict(ldo=1020), SHAPE),
                       (dict(ty=1, ldq=1026), SHAPE), (dict(ldk=1 << 41), SHAPE), (dict(q=at(8) + 8), ALIGN), (dict(k=at(8) + 2), ALIGN),
                       (dict(v=at(8) + 4), ALIGN), (dict(out=at(8) + 8), ALIGN), (dict(rot=32), SHAPE), (dict(rot=192), SHAPE),
                       (dict(rot=-64), SHAPE), (dict(cos=None), NULL), (dict(sin=None), NULL), (dict(cos=at(1) + 4), ALIGN),
                       (dict(sin=at(1) + 8), ALIGN), (dict(pos=at(1) + 2), ALIGN), (dict(angles=0), SHAPE), (dict(angles=1 << 41), SHAPE)]:
        assert append(L, **more) == code, more


def test_gather_validation(L):
    for more, code in [(dict(k=None, v=None), NULL), (dict(ldk=504), SHAPE), (dict(ldv=516), SHAPE), (dict(k=at(1) + 8), ALIGN), (dict(v=at(1) + 2), ALIGN)]:
        assert gather(L, **more) == code, more


def test_attn_validation(L):
    need = L.snipkv_attn_workspace(5, 3, 8, 4, 128)
    assert need > 0
    for more, code in [(dict(q=None), NULL), (dict(out=None), NULL), (dict(heads=6), SHAPE), (dict(heads=0), SHAPE), (dict(ldq=1016), SHAPE),
                       (dict(ldo=1028), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(scale=3e38), SHAPE),
                       (dict(scale=float("nan")), SHAPE), (dict(window=-1), SHAPE), (dict(q=at(1) + 8), ALIGN), (dict(out=at(1) + 2), ALIGN),
                       (dict(lse=at(1) + 2), ALIGN), (dict(ws=at(1) + 8), ALIGN), (dict(ws=None), WORKSPACE), (dict(n=need - 1), WORKSPACE),
                       (dict(heads=1024, c=cache(heads=1), tokens=1 << 20, ldq=1 << 17, ldo=1 << 17), SHAPE)]:
        assert attn(L, **more) == code, more


def test_workspace_sizes(L):
    w = L.snipkv_attn_workspace
    assert w(1, 1, 1, 1, 64) > 0 and w(1, 1, 64, 8, 128) == w(4096, 16, 64, 8, 128) > 0
    for bad in [(0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 1, 0, 1, 64), (1, 1, 1, 0, 64), (1, 1, 3, 2, 64), (1, 1, 1, 1, 96),
                ((1 << 20) + 1, 1, 1, 1, 64), (1, (1 << 20) + 1, 1, 1, 64), (1, 1, 1025, 1, 64), (1 << 20, 1, 1024, 1, 64),
                (1 << 20, 1 << 20, 1024, 1024, 64)]:
        assert w(*bad) == 0, bad


def test_cache_shapes():
    for fmt, block in ((S.NVFP4, 16), (S.MXFP4, 32)):
        for dim in kv.HEAD_DIMS:
            k, ks, v, vs = kv.cache_shapes(fmt, 3, 32, 2, dim)
            size = lambda s: s[0] * s[1] * s[2] * s[3] * s[4] * (s[5] if len(s) > 5 else 1)  # noqa: E731
            assert size(k) == size(v) == 3 * 32 * 2 * dim // 2 and size(ks) == size(vs) == 3 * 32 * 2 * dim // block
    for bad in [(S.FP8, 1, 16, 1, 64), (S.NVFP4, 1, 24, 1, 64), (S.NVFP4, 1, 8, 1, 64), (S.NVFP4, 1, 8192, 1, 64), (S.MXFP4, 1, 16, 1, 80)]:
        with pytest.raises(ValueError):
            kv.cache_shapes(*bad)
