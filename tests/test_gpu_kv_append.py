"""snipkv_append and snipkv_gather: rotated queries, codes and scales bit for
bit against the oracle's rotation and quantizer; everything else untouched."""
import numpy as np
import pytest
import torch

import sub_byte_mixed_amd as S
from kv_common import TEXP, Paged, make_cache, quantized, tokens_view
from oracle import formats as F
from oracle import kv as OK
from ops_common import BF, F32, Guarded, f64, rand, say, strided

pytestmark = pytest.mark.gpu
FORMATS = [S.NVFP4, S.MXFP4]


def angles(n, rot, seed=9):
    g = torch.Generator().manual_seed(seed)
    a = 20.0 * torch.rand((n, rot // 2), generator=g, dtype=torch.float64)
    return a.cos().float(), a.sin().float()


def expected(P, q, k, v, cos, sin, inter, pos=None):
    """(q in bf16, token-major codes and scales of k and v per row) from the oracle."""
    n, dim = P.rows, P.dim
    at = np.concatenate([P.positions(b) for b in range(len(P.lens))]) if pos is None else pos
    q, k, v = (None if t is None else t.float().numpy()[:n].reshape(n, -1, dim) for t in (q, k, v))
    if cos is not None:
        i = np.clip(at, 0, cos.shape[0] - 1)
        c, s = cos.numpy()[i], sin.numpy()[i]
        q = None if q is None else OK.rotate(q, c, s, inter)
        k = None if k is None else OK.rotate(k, c, s, inter)
    enc = [None if x is None else quantized(x.reshape(-1, dim), P.fmt, e) for x, e in ((k, TEXP[0]), (v, TEXP[1]))]
    return (None if q is None else torch.from_numpy(q.reshape(n, -1)).to(BF)), enc


def snapshot(cache):
    return [t.clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]


def check_cache(P, before, enc):
    """The rows' tokens hold enc, every other byte what it held before."""
    c = P.cache
    bufs = (c.k_codes, c.k_scales, c.v_codes, c.v_scales)
    for i, (t, old) in enumerate(zip(bufs, before)):
        keys = i < 2
        want = tokens_view(old, keys).copy()
        e = enc[i // 2]
        if e is not None:
            rows = e[i % 2].reshape(P.rows, P.heads, -1)
            for b in range(len(P.lens)):
                for j, p in enumerate(P.positions(b)):
                    if p < 0 or p >= P.table.shape[1] * P.page:
                        continue
                    page = int(P.table[b, p // P.page])
                    if 0 <= page < c.pages:
                        want[page, :, p % P.page] = rows[P.cu[b] + j]
        got = tokens_view(t, keys)
        bad = np.argwhere(got != want)
        assert not bad.size, (i, len(bad), bad[:4].tolist(), got[tuple(bad[0])], want[tuple(bad[0])])


CASES = [  # dim, heads, query heads, page, lens, new
    (64, 1, 1, 16, [1], [1]),
    (64, 4, 32, 64, [700], [1]),
    (128, 8, 64, 32, [5, 33, 1, 64, 17], [1, 1, 1, 1, 1]),
    (128, 3, 9, 16, [40, 7, 129], [37, 7, 2]),
    (256, 2, 6, 128, [131, 20], [131, 3]),
    (64, 5, 5, 16, [19, 0, 80], [19, 0, 33]),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append(fmt, dtype, case):
    dim, heads, hq, page, lens, new = CASES[case]
    say("append", fmt, dtype, case)
    P = Paged(fmt, dim, heads, page, lens, new, seed=case, one_each=all(n == 1 for n in new))
    for rot in sorted({0, 64, dim}):
        for inter in (False, True):
            q, k, v = (rand((P.rows, h * dim), dtype, 3 * case + i, s) for i, (h, s) in enumerate(((hq, 1.0), (heads, 2.0), (heads, 0.3))))
            cos, sin = angles(max(lens) + 1, rot) if rot else (None, None)
            before = snapshot(P.cache)
            dev = [None if t is None else t.cuda() for t in (cos, sin)]
            got = S.kv_append(strided(k, 8), strided(v, 16), P.cache, P.batch, q=strided(q, 8), cos=dev[0], sin=dev[1], interleaved=inter)
            want, enc = expected(P, q, k, v, cos, sin, inter)
            assert torch.equal(got.cpu(), want), (rot, inter)
            check_cache(P, before, enc)


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_product_in_place_and_without_queries(fmt):
    dim, heads, hq = 128, 2, 4
    P = Paged(fmt, dim, heads, 16, [50, 3], [20, 3])
    qkv = rand((P.rows, (hq + 2 * heads) * dim), BF, 1)
    cos, sin = angles(64, dim)
    a, b = hq * dim, (hq + heads) * dim
    want, enc = expected(P, qkv[:, :a], qkv[:, a:b], qkv[:, b:], cos, sin, False)
    d = qkv.cuda()
    before = snapshot(P.cache)
    S.kv_append(d[:, a:b], d[:, b:], P.cache, P.batch, q=d[:, :a], cos=cos.cuda(), sin=sin.cuda(), q_out=d[:, :a])
    assert torch.equal(d[:, :a].cpu(), want) and torch.equal(d[:, a:].cpu(), qkv[:, a:])
    check_cache(P, before, enc)
    for t, old in zip((P.cache.k_codes, P.cache.k_scales, P.cache.v_codes, P.cache.v_scales), before):
        t.copy_(old)
    assert S.kv_append(d[:, a:b], d[:, b:], P.cache, P.batch, cos=cos.cuda(), sin=sin.cuda()) is None
    check_cache(P, before, enc)
    after = snapshot(P.cache)
    q = qkv[:, :a].cuda()
    got = S.kv_append(None, None, P.cache, P.batch, q=q, cos=cos.cuda(), sin=sin.cuda())
    assert torch.equal(got.cpu(), want) and all(torch.equal(x, y) for x, y in zip(after, snapshot(P.cache)))


def test_positions_of_the_callers_and_beyond_the_angles():
    P = Paged(S.NVFP4, 64, 2, 16, [30], [9])
    q, k, v = (rand((9, 128), F32, i) for i in range(3))
    cos, sin = angles(25, 64)
    for pos in (None, np.array([0, 24, 25, 1000, -1, 2 ** 31 - 1, -2 ** 31, 3, 3], np.int32)):
        before = snapshot(P.cache)
        got = S.kv_append(k.cuda(), v.cuda(), P.cache, P.batch, q=q.cuda(), cos=cos.cuda(), sin=sin.cuda(),
                          pos=None if pos is None else torch.from_numpy(pos).cuda())
        want, enc = expected(P, q, k, v, cos, sin, False, None if pos is None else pos.astype(np.int64))
        assert torch.equal(got.cpu(), want)
        check_cache(P, before, enc)


@pytest.mark.parametrize("fmt", FORMATS)
def test_unmapped_places_and_rows_of_nobody(fmt):
    """Pages that the table does not name, positions before 0 and behind the table, rows behind the last sequence:
    nothing is written, and the queries of the rows that belong to a sequence are rotated all the same."""
    P = Paged(fmt, 64, 2, 16, [40, 5, 70], [30, 9, 2], unmapped=[(0, 1), (2, 4)])
    P.batch = S.KVBatch(P.batch.table[:, :4], P.batch.lens, P.batch.cu)     # 64 positions: sequence 2 runs over
    P.table = P.table[:, :4]
    rows = P.rows + 6
    q, k, v = (rand((rows, 128), BF, i) for i in range(3))
    cos, sin = angles(80, 64)
    out = Guarded(rows, 128, BF)
    before = snapshot(P.cache)
    S.kv_append(k.cuda(), v.cuda(), P.cache, P.batch, q=q.cuda(), cos=cos.cuda(), sin=sin.cuda(), q_out=out.t)
    want, enc = expected(P, q, k, v, cos, sin, False)
    check_cache(P, before, enc)
    assert torch.equal(out.t[:P.rows].cpu(), want) and bool((out.t[P.rows:] == 7.0).all()) and out.intact()
    gk, gv = Guarded(rows, 128, BF), Guarded(rows, 128, BF)
    S.kv_gather(P.cache, P.batch, k=gk.t, v=gv.t)
    assert bool((gk.t[P.rows:] == 7.0).all()) and gk.intact() and gv.intact()
    for b in range(3):
        for j, p in enumerate(P.positions(b)):
            if p < 0 or p >= 64 or (b, p // 16) in ((0, 1), (2, 4)):
                assert not gk.t[P.cu[b] + j].any() and not gv.t[P.cu[b] + j].any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_gather(fmt, dim):
    """The float64 values of the stored bytes, which bf16 holds exactly here."""
    say("gather", fmt, dim)
    P = Paged(fmt, dim, 3, 16, [37, 1, 16], [37, 1, 16], seed=dim)
    k, v = S.kv_gather(P.cache, P.batch, P.rows)
    for b in range(3):
        wk, wv = P.values(b)
        r = slice(P.cu[b], P.cu[b + 1])
        for got, want in ((k, wk), (v, wv)):
            assert np.array_equal(f64(got[r]).reshape(P.lens[b], 3, dim), want.transpose(1, 0, 2))


@pytest.mark.parametrize("fmt", FORMATS)
def test_values_at_the_ends(fmt):
    """Zeros, infinities, NaN, the largest and smallest numbers, a block of nothing but NaN."""
    P = Paged(fmt, 64, 1, 16, [8], [8])
    x = rand((8, 64), F32, 5)
    x[0] = 0.0
    x[1, 3], x[1, 40] = float("inf"), float("-inf")
    x[2, 5] = float("nan")
    x[3] = float("nan")
    x[4] *= 1e38
    x[5] *= 1e-42
    x[6, ::2] = -0.0
    x[7] = float("inf")
    before = snapshot(P.cache)
    S.kv_append(x.cuda(), x.cuda(), P.cache, P.batch)
    fin = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).numpy()
    enc = []
    for e in TEXP:
        codes, scales = quantized(fin, fmt, e)
        n = F.unpack_nibbles(codes)
        n = np.where(np.isposinf(x.numpy()), 7, np.where(np.isneginf(x.numpy()), 15, n))
        if fmt == S.NVFP4:                              # a block whose scale is zero has no magnitude
            n = np.where(np.repeat(scales == 0, 16, axis=1), n & 8, n)
        else:
            zero = np.repeat((np.abs(fin).reshape(8, -1, 32).max(axis=2) == 0), 32, axis=1)
            n = np.where(zero, n & 8, n)
        n = np.where(np.isnan(x.numpy()), 0, n)
        enc.append((F.pack_nibbles(n.astype(np.uint8)), scales))
    check_cache(P, before, enc)


def test_many_sequences_and_tokens():
    """More sequences than a wave looks up at once, some without tokens; more rows than waves of a launch."""
    new = [(7 * b) % 4 for b in range(5000)]
    new[4999] = 2
    P = Paged(S.NVFP4, 64, 1, 16, [n if n else 3 for n in new], new, seed=3)
    k, v = rand((P.rows, 64), BF, 1), rand((P.rows, 64), BF, 2)
    before = snapshot(P.cache)
    S.kv_append(k.cuda(), v.cuda(), P.cache, P.batch)
    _, enc = expected(P, None, k, v, None, None, False)
    check_cache(P, before, enc)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,dtype", [(64, BF), (64, F32), (128, F32), (128, BF), (256, F32)])
def test_long_calls(fmt, dim, dtype):
    """Calls of many waves, which take four tokens each, against the same tokens in short calls: sequences that
    begin and end anywhere, positions that are not multiples of four, pages that are not mapped, rows of nobody."""
    heads, hq, page = 8192 // dim, 16384 // dim, 16
    lens, new = [700, 1203, 7, 66, 2, 0, 301, 33], [700, 1001, 5, 66, 1, 0, 298, 30]
    say("append long", fmt, dim, dtype)
    P = Paged(fmt, dim, heads, page, lens, new, seed=dim, unmapped=[(0, 3), (1, 20), (1, 21), (3, 0)])
    rows = P.rows + 13
    q, k, v = (rand((rows, h * dim), dtype, i).cuda() for i, h in enumerate((hq, heads, heads)))
    cos, sin = (t.cuda() for t in angles(1300, 64))
    start = snapshot(P.cache)
    out = Guarded(rows, hq * dim, BF)
    S.kv_append(k, v, P.cache, P.batch, q=q, cos=cos, sin=sin, interleaved=dim == 64, q_out=out.t)
    got = snapshot(P.cache)
    gathered = [torch.full((rows, heads * dim), 7.0, dtype=BF, device="cuda") for _ in range(2)]
    S.kv_gather(P.cache, P.batch, k=gathered[0], v=gathered[1])
    for t, old in zip((P.cache.k_codes, P.cache.k_scales, P.cache.v_codes, P.cache.v_scales), start):
        t.copy_(old)
    want, parts = torch.full_like(out.t, 7.0), [torch.full_like(gathered[0], 7.0) for _ in range(2)]
    for b in range(len(lens)):
        for a in range(0, new[b], 150):
            n = min(150, new[b] - a)
            r = slice(int(P.cu[b]) + a, int(P.cu[b]) + a + n)
            batch = S.KVBatch(P.batch.table[b:b + 1], torch.tensor([lens[b] - new[b] + a + n], dtype=torch.int32, device="cuda"),
                              torch.tensor([0, n], dtype=torch.int32, device="cuda"))
            want[r] = S.kv_append(k[r], v[r], P.cache, batch, q=q[r], cos=cos, sin=sin, interleaved=dim == 64)
            for t, p in zip(S.kv_gather(P.cache, batch, n), parts):
                p[r] = t
    assert torch.equal(out.t, want) and out.intact()
    assert all(torch.equal(a, b) for a, b in zip(got, snapshot(P.cache)))
    assert all(torch.equal(a, b) for a, b in zip(gathered, parts))


def test_other_stream():
    P = Paged(S.NVFP4, 64, 2, 16, [40], [40])
    k, v, q = (rand((40, 128), BF, i).cuda() for i in range(3))
    want = S.kv_append(k, v, P.cache, P.batch, q=q)
    stored = S.kv_gather(P.cache, P.batch, 40)
    s = torch.cuda.Stream()
    for t in (P.cache.k_codes, P.cache.v_codes):
        t.zero_()
    torch.cuda.synchronize()
    got = S.kv_append(k, v, P.cache, P.batch, q=q, stream=s)
    again = S.kv_gather(P.cache, P.batch, 40, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(again, stored))
