"""The operators' binding (sub_byte_mixed_amd/ops.py) without a GPU: the calls
on CPU stand-ins for GPU tensors, with the library's launching entries stubbed
and its sizers real."""
import contextlib
import os
import weakref

import pytest
import torch

import sub_byte_mixed_amd as S
from sub_byte_mixed_amd import ops

BF, F32 = torch.bfloat16, torch.float32
HERE = -1                                              # what get_device() says of a CPU tensor


class Library:
    """libsnip with its launching entries replaced by `launch(name, args)`."""

    def __init__(self, real, launch):
        self.real, self.launch = real, launch

    def __getattr__(self, name):
        if name.startswith("snipop_") and not name.endswith("_workspace"):
            return lambda *a: self.launch(name, a)
        return getattr(self.real, name)


class Stand:
    """CPU tensors taken for those of device -1; `made`: what was allocated."""

    def __init__(self, monkeypatch):
        if not os.path.exists(S.LIB_PATH):
            from sub_byte_mixed_amd import build
            build.build()
        self.made, self.calls, self.during = [], [], None
        real, empty, zeros = S.lib(), torch.empty, torch.zeros

        def cpu(make):
            def f(*a, device=None, **k):
                t = make(*a, device="cpu" if device == HERE else device, **k)
                self.made.append((weakref.ref(t), t.data_ptr(), t.nbytes))
                return t
            return f

        def launch(name, args):
            self.calls.append((name, args))
            if self.during:
                self.during(name, args)
            return 0
        monkeypatch.setattr(torch, "empty", cpu(empty))
        monkeypatch.setattr(torch, "zeros", cpu(zeros))
        monkeypatch.setattr(S, "lib", lambda: Library(real, launch))
        monkeypatch.setattr(ops, "_device", lambda t, fn: t.get_device())
        monkeypatch.setattr(ops, "_current_device", lambda: HERE)
        monkeypatch.setattr(ops, "_current_stream", lambda dev: 0)

    def alive(self, address, size):
        return any(r() is not None and p == address and n >= size for r, p, n in self.made)


@pytest.fixture
def stand(monkeypatch):
    return Stand(monkeypatch)


@pytest.mark.parametrize("fmt", [S.FP8, S.NVFP4, S.MXFP4])
def test_workspace_lives_until_the_launches_are_enqueued(stand, fmt):
    """A workspace that a call allocates for itself is still held when the
    library runs: memory given back earlier may be another call's by then."""
    def during(name, args):
        ws, size = args[-3:-1]
        assert ws and size and stand.alive(ws, size), name
    stand.during = during
    x, gamma = torch.ones((4, 64), dtype=BF), torch.ones(64, dtype=BF)
    S.rmsnorm_fwd(x, gamma, out_fmt=fmt)
    S.rmsnorm_fwd(x, gamma, with_y=False, with_rstd=False, out_fmt=fmt)
    S.swiglu_fwd(x, x, out_fmt=fmt)
    S.swiglu_fwd(x, x, with_y=False, q=S.QuantizedTensor(fmt, 4, 64, HERE))
    if fmt != S.MXFP4:                                 # to find the maximum alone
        S.rmsnorm_fwd(x, gamma, out_fmt=fmt, with_stats=False)
        S.swiglu_fwd(x, x, out_fmt=fmt, with_stats=False)
    assert len(stand.calls) == (4 if fmt == S.MXFP4 else 6)


def test_workspace_of_the_backward_norm_lives_as_long(stand):
    def during(name, args):
        assert stand.alive(*args[-3:-1]), name
    stand.during = during
    x = torch.ones((4, 64), dtype=BF)
    S.rmsnorm_bwd(x, x, torch.ones(64, dtype=BF), torch.ones(4))
    assert len(stand.calls) == 1


class Streams:
    """torch.cuda's streams for the stand-ins: `stream(s)` makes s the current
    one and its device the current device, as torch's does."""

    class Stream:
        def __init__(self, handle, device_index):
            self.cuda_stream, self.device_index = handle, device_index
            self.device = torch.device("cpu")

    class ExternalStream(Stream):
        pass

    def __init__(self, monkeypatch):
        self.device, self.current = HERE, {HERE: 0, 3: 30}
        monkeypatch.setattr(torch.cuda, "Stream", self.Stream)
        monkeypatch.setattr(torch.cuda, "ExternalStream", self.ExternalStream)
        monkeypatch.setattr(torch.cuda, "default_stream", lambda dev: self.Stream(0, dev))
        monkeypatch.setattr(torch.cuda, "stream", lambda s: self.switch(s.device_index, s.cuda_stream))
        monkeypatch.setattr(torch.cuda, "device", lambda dev: self.switch(dev, self.current[dev]))
        monkeypatch.setattr(ops, "_current_device", lambda: self.device)
        monkeypatch.setattr(ops, "_current_stream", lambda dev: self.current[dev])

    @contextlib.contextmanager
    def switch(self, device, handle):
        was = self.device, dict(self.current)
        self.device, self.current[device] = device, handle
        yield
        self.device, self.current = was


def calls_with(stream):
    """Each entry of the binding on `stream`."""
    x, gamma, rstd = torch.ones((4, 64), dtype=BF), torch.ones(64, dtype=BF), torch.ones(4)
    w = S.QuantizedTensor(S.NVFP4, 8, 64, HERE)
    return [lambda: S.rmsnorm_fwd(x, gamma, out_fmt=S.FP8, stream=stream), lambda: S.rmsnorm_bwd(x, x, gamma, rstd, stream=stream),
            lambda: S.swiglu_fwd(x, x, stream=stream), lambda: S.swiglu_bwd(x, x, x, stream=stream),
            lambda: S.qgemv(x, w, stream=stream)]


def test_a_stream_of_another_device_is_refused(stand, monkeypatch):
    streams = Streams(monkeypatch)
    for call in calls_with(streams.Stream(31, 3)):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert not stand.calls and streams.device == HERE


def test_streams_and_handles_reach_the_library(stand, monkeypatch):
    """A stream, its handle, the default stream's handle, and any object with
    the attribute that the package's other calls read."""
    class Foreign:
        cuda_stream = 77
    streams = Streams(monkeypatch)
    for stream, handle in ((streams.Stream(11, HERE), 11), (12, 12), (0, 0), (Foreign(), 77)):
        stand.calls.clear()
        for call in calls_with(stream):
            call()
        assert [a[-1] for _, a in stand.calls] == [handle] * 5
    assert streams.device == HERE and streams.current[HERE] == 0


def test_tensors_of_another_device_run_there(stand, monkeypatch):
    streams = Streams(monkeypatch)
    streams.device = 3
    stand.calls.clear()
    for call in calls_with(None):
        call()
    assert [a[-1] for _, a in stand.calls] == [0] * 5 and streams.device == 3


def test_qgemv_weights_beyond_a_grid_are_refused(stand):
    """2^40 weights are more than a card holds; within them every launch's
    grid has fewer than 2^32 threads a dimension."""
    import ctypes
    at = 0x7F0000000000                                # made up, never touched
    L = S.lib().real

    def gemv(n, k):
        w = S.QTensorDesc(S.NVFP4, 0, n, k, at, at, at)
        return L.snipop_qgemv(at, k, 1, ctypes.byref(w), at, 0, n, None)
    assert gemv(1 << 31, 544) == -2 and "2^40" in L.snip_last_error().decode()
    assert gemv((1 << 15) + 1, 1 << 25) == -2


class Elsewhere:
    """What the binding asks of a device tensor, on device 3."""
    is_cuda, dtype = True, F32
    data_ptr, numel, get_device, is_contiguous = lambda s: 4096, lambda s: 1, lambda s: 3, lambda s: True


def test_a_maximum_on_another_device_is_refused(stand):
    x, gamma = torch.ones((4, 64), dtype=BF), torch.ones(64, dtype=BF)
    record = S.StatsAmax.__new__(S.StatsAmax)
    record.stats, record.i = Elsewhere(), 0
    for amax in (Elsewhere(), record):
        with pytest.raises(ValueError, match="amax"):
            S.rmsnorm_fwd(x, gamma, out_fmt=S.FP8, amax=amax)
        with pytest.raises(ValueError, match="amax"):
            S.swiglu_fwd(x, x, out_fmt=S.NVFP4, amax=amax)
    assert not stand.calls


def test_no_workspace_for_shapes_that_the_calls_refuse(stand):
    L = S.lib()
    for rows in ((1 << 40) + 1, (1 << 63) - 1):
        assert L.snipop_rmsnorm_bwd_workspace(rows, 64) == 0
        assert L.snipop_rmsnorm_fwd_workspace(rows, 64, S.FP8) == 0
        assert L.snipop_swiglu_fwd_workspace(rows, 64, S.FP8) == 0
    assert L.snipop_swiglu_fwd_workspace(4, (1 << 31) + 16, S.FP8) == 0
    assert L.snipop_swiglu_fwd_workspace(4, 1 << 31, S.FP8) > 0
