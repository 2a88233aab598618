"""The cache's binding (sub_byte_mixed_amd/kv.py) without a GPU: the calls on
CPU stand-ins for GPU tensors, with the library's launching entries stubbed and
its sizer real."""
import contextlib
import ctypes
import os

import pytest
import torch

import sub_byte_mixed_amd as S
from sub_byte_mixed_amd import kv, ops

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
HERE = -1                                              # what get_device() says of a CPU tensor


class Stand:
    def __init__(self, monkeypatch):
        if not os.path.exists(S.LIB_PATH):
            from sub_byte_mixed_amd import build
            build.build()
        real, stand = S.lib(), self
        self.calls = []

        class Library:
            def __getattr__(self, name):
                if name.startswith("snipkv_") and not name.endswith("_workspace"):
                    return lambda *a: stand.calls.append((name, a)) or 0
                return getattr(real, name)
        monkeypatch.setattr(S, "lib", lambda: Library())
        monkeypatch.setattr(kv, "_CPU", None)
        monkeypatch.setattr(ops, "_current_device", lambda: HERE)
        monkeypatch.setattr(ops, "_current_stream", lambda dev: 77)


@pytest.fixture
def stand(monkeypatch):
    return Stand(monkeypatch)


def make(fmt=S.NVFP4, pages=4, page=32, heads=2, dim=64, seqs=3, new=(2, 0, 3)):
    cache = S.KVCache.empty(fmt, pages, page, heads, dim, "cpu", texp=(-3, 2))
    table = torch.zeros((seqs, 5), dtype=I32)[:, :4]
    cu = torch.tensor([0, *torch.tensor(new).cumsum(0).tolist()], dtype=I32) if new else None
    return cache, S.KVBatch(table, torch.ones(seqs, dtype=I32), cu)


def test_descriptors(stand):
    cache, batch = make()
    d, b = cache._desc, batch._desc
    assert (d.format, d.page_size, d.kv_heads, d.head_dim, d.pages) == (S.NVFP4, 32, 2, 64, 4)
    assert (d.k_codes, d.v_scales, d.texp) == (cache.k_codes.data_ptr(), cache.v_scales.data_ptr(), cache.texp.data_ptr())
    assert cache.texp.tolist() == [-3, 2]
    assert (b.table, b.table_ld, b.max_pages, b.lens, b.cu, b.seqs) == (batch.table.data_ptr(), 5, 4, batch.lens.data_ptr(), batch.cu.data_ptr(), 3)
    mx = S.KVCache.empty(S.MXFP4, 1, 16, 1, 256, "cpu")
    assert mx.texp is None and mx._desc.texp is None and mx.page_size == 16 and mx.head_dim == 256
    assert S.KVBatch(torch.zeros((1, 7), dtype=I32), torch.ones(1, dtype=I32))._desc.table_ld == 7


def test_cache_refusals(stand):
    good = make()[0]
    bufs = [good.k_codes, good.k_scales, good.v_codes, good.v_scales]
    for i in range(4):
        for bad in (bufs[i].to(torch.int8), bufs[i][..., :-1], bufs[i][:1].expand_as(bufs[i])):
            with pytest.raises(ValueError):
                S.KVCache(S.NVFP4, *bufs[:i], bad, *bufs[i + 1:], good.texp)
    for texp in (None, good.texp.long(), good.texp[:1]):
        with pytest.raises(ValueError):
            S.KVCache(S.NVFP4, *bufs, texp)
    with pytest.raises(ValueError):
        S.KVCache(S.FP8, *bufs, good.texp)
    with pytest.raises(ValueError):
        S.KVCache(S.MXFP4, *bufs)                      # another number of scales
    with pytest.raises(ValueError):
        S.KVCache(S.NVFP4, bufs[0].flatten(), *bufs[1:], good.texp)


def test_batch_refusals(stand):
    t, n = torch.zeros((3, 4), dtype=I32), torch.ones(3, dtype=I32)
    for bad in [(t.long(), n), (t[0], n), (t.t().contiguous().t(), n), (t, n.long()), (t, n[:2]), (t, n, torch.zeros(3, dtype=I32)),
                (t, n, torch.zeros(4))]:
        with pytest.raises(ValueError):
            S.KVBatch(*bad)


def test_append_arguments(stand):
    cache, batch = make()
    qkv = torch.zeros((5, (4 + 2 + 2) * 64), dtype=F32)
    q, k, v = qkv[:, :256], qkv[:, 256:384], qkv[:, 384:]
    cos = torch.zeros((9, 32))
    pos = torch.zeros(5, dtype=I32)
    out = S.kv_append(k, v, cache, batch, q=q, cos=cos, sin=cos, interleaved=True, pos=pos)
    assert out.dtype == BF and out.shape == (5, 256)
    name, a = stand.calls[-1]
    assert name == "snipkv_append"
    assert a[:15] == (q.data_ptr(), 512, 4, k.data_ptr(), 512, v.data_ptr(), 512, 1, 5, cos.data_ptr(), cos.data_ptr(), 9, 64, True,
                      pos.data_ptr())
    assert a[15] is cache.ref and a[16] is batch.ref and a[17:] == (out.data_ptr(), 256, 77)
    assert S.kv_append(k, v, cache, batch) is None
    a = stand.calls[-1][1]
    assert a[0] is None and a[2] == 0 and a[9] is None and a[12] == 0 and a[17] is None
    buf = torch.zeros((5, 256), dtype=BF)
    assert S.kv_append(None, None, cache, batch, q=buf, q_out=buf) is buf
    a = stand.calls[-1][1]
    assert a[0] == a[17] == buf.data_ptr() and a[3] is None and a[5] is None and a[7] == 0


def test_append_refusals(stand):
    cache, batch = make()
    k = v = torch.zeros((5, 128), dtype=BF)
    q, cos = torch.zeros((5, 256), dtype=BF), torch.zeros((9, 32))
    for a, more in [((None, v), {}), ((k, None), {}), ((None, None), {}), ((k.half(), v.half()), {}), ((k, v.float()), {}),
                    ((k, v), dict(q=q.float())), ((k, v), dict(q=q[:4])), ((k, v[:4]), {}), ((k[:, :64], v), {}), ((k, v[:, :64]), {}),
                    ((k, v), dict(q=q[:, :200])), ((k, v), dict(q_out=q)), ((k, v), dict(q=q, q_out=q.float())),
                    ((k, v), dict(q=q, q_out=q[:, :128])), ((k, v), dict(cos=cos)), ((k, v), dict(sin=cos)),
                    ((k, v), dict(cos=cos, sin=cos[:, :16])), ((k, v), dict(cos=cos.double(), sin=cos.double())),
                    ((k, v), dict(cos=cos.t(), sin=cos.t())), ((k, v), dict(pos=torch.zeros(4, dtype=I32))),
                    ((k, v), dict(pos=torch.zeros(5, dtype=torch.int64))), ((k[0], v[0]), {}), ((k.t(), v.t()), {}),
                    (([1], v), {})]:
        with pytest.raises(ValueError):
            S.kv_append(*a, cache, batch, **more)
    assert not stand.calls


def test_attn_arguments(stand):
    cache, batch = make()
    q = torch.zeros((5, 512), dtype=BF)[:, :256]
    out, lse = S.kv_attn(q, cache, batch, window=9, with_lse=True)
    name, a = stand.calls[-1]
    assert name == "snipkv_attn" and out.shape == (5, 256) and out.dtype == BF and lse.shape == (5, 4) and lse.dtype == F32
    assert a[:4] == (q.data_ptr(), 512, 4, 5) and a[4] is cache.ref and a[5] is batch.ref
    assert a[6] == pytest.approx(0.125) and a[7] == 9 and a[8:11] == (out.data_ptr(), 256, lse.data_ptr())
    assert a[12] == S.lib().snipkv_attn_workspace(5, 3, 4, 2, 64) and a[13] == 77
    ws = torch.zeros(a[12], dtype=torch.uint8)
    got, none = S.kv_attn(q, cache, batch, scale=2.0, out=q, ws=ws)
    a = stand.calls[-1][1]
    assert got is q and none is None and a[6] == 2.0 and a[7] == 0 and a[10:13] == (None, ws.data_ptr(), ws.nbytes)
    one = make(seqs=1, new=None)[1]
    S.kv_attn(torch.zeros((1, 99 * 64), dtype=BF)[:, :64], cache, one)
    assert stand.calls[-1][1][1] == 64                 # one row: its stride says nothing


def test_attn_refusals(stand):
    cache, batch = make()
    q = torch.zeros((5, 256), dtype=BF)
    for a, more in [((q.float(),), {}), ((q[:, :100],), {}), ((q[0],), {}), ((q.t(),), {}), ((q,), dict(out=q.float())), ((q,), dict(out=q[:4])),
                    ((q,), dict(lse=torch.zeros(5, 3))), ((q,), dict(lse=torch.zeros(5, 4, dtype=torch.float64))),
                    ((q,), dict(lse=torch.zeros(4, 5).t())), ((q,), dict(ws=torch.zeros(99, 9, dtype=torch.uint8)[:, ::2])),
                    ((q[:, :0],), {})]:
        with pytest.raises(ValueError):
            S.kv_attn(*a, cache, batch, **more)
    assert not stand.calls


def test_gather_arguments(stand):
    cache, batch = make()
    k, v = S.kv_gather(cache, batch, 5)
    name, a = stand.calls[-1]
    assert name == "snipkv_gather" and k.shape == v.shape == (5, 128) and k.dtype == BF
    assert a[0] is cache.ref and a[1] is batch.ref and a[2:] == (5, k.data_ptr(), 128, v.data_ptr(), 128, 77)
    assert S.kv_gather(cache, make(new=None)[1])[0].shape == (3, 128)
    assert S.kv_gather(cache, batch, k=k)[0] is k
    for more in [dict(k=k.float()), dict(v=v[:, :64]), dict(k=k, v=v[:3])]:
        with pytest.raises(ValueError):
            S.kv_gather(cache, batch, **more)


def test_places(stand):
    """The cache and the batch on different GPUs, and matrices elsewhere than both."""
    cache, batch = make()
    other = make()[1]
    other.device = 3
    q = torch.zeros((5, 256), dtype=BF)
    for call in (lambda b: S.kv_attn(q, cache, b), lambda b: S.kv_append(q[:, :128], q[:, :128], cache, b), lambda b: S.kv_gather(cache, b, 5)):
        with pytest.raises(ValueError):
            call(other)
    assert not stand.calls


def test_streams_and_devices(stand, monkeypatch):
    """Another device than the current one, and stream=: the call is made with them current."""
    cache, batch = make()
    current = [3]

    @contextlib.contextmanager
    def switch(dev):
        was, current[0] = current[0], dev
        yield
        current[0] = was
    monkeypatch.setattr(ops, "_current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", switch)
    S.kv_attn(torch.zeros((5, 256), dtype=BF), cache, batch)
    assert len(stand.calls) == 1 and current == [3]

    class Stream:
        device_index, cuda_stream = 5, 12
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    with pytest.raises(ValueError):                    # a stream of another GPU
        S.kv_attn(torch.zeros((5, 256), dtype=BF), cache, batch, stream=Stream())


def test_the_workspace_is_held_until_the_call_has_returned(stand, monkeypatch):
    cache, batch = make()
    q = torch.zeros((5, 256), dtype=BF)
    made = []
    real = torch.Tensor.new_empty
    monkeypatch.setattr(torch.Tensor, "new_empty", lambda self, *a, **k: made.append(real(self, *a, **k)) or made[-1])
    S.kv_attn(q, cache, batch)
    a = stand.calls[-1][1]
    ws = [t for t in made if t.data_ptr() == a[11]]
    assert len(ws) == 1 and ws[0].nbytes == a[12]


def test_cpu_tensors_are_refused():
    cache, batch = make()
    q = torch.zeros((5, 256), dtype=BF)
    for call in (lambda: S.kv_attn(q, cache, batch), lambda: S.kv_append(q[:, :128], q[:, :128], cache, batch), lambda: S.kv_gather(cache, batch, 5)):
        with pytest.raises(ValueError):
            call()


def test_descriptor_fields_keep_the_tensors_alive():
    cache, batch = make()
    assert all(t is not None for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales, cache.texp, batch.table, batch.lens, batch.cu))
    assert ctypes.sizeof(kv.CacheDesc) == 64 and ctypes.sizeof(kv.BatchDesc) == 48
