"""The tensors of a KVCache and a KVBatch, whose addresses the library was given:
written into in place they are followed; replaced by others they would not be,
so that is refused. On CPU tensors: no call is made."""
import pytest
import torch

import sub_byte_mixed_amd as S

I32 = torch.int32


def batch(cu=True):
    return S.KVBatch(torch.zeros((2, 3), dtype=I32), torch.tensor([4, 5], dtype=I32), torch.tensor([0, 1, 3], dtype=I32) if cu else None)


@pytest.mark.parametrize("name", ["table", "lens", "cu"])
def test_a_batch_keeps_its_tensors(name):
    b = batch()
    old = getattr(b, name)
    with pytest.raises(AttributeError, match=name):
        setattr(b, name, old + 1)
    assert getattr(b, name) is old
    with pytest.raises(AttributeError, match="cu"):
        batch(cu=False).cu = torch.tensor([0, 1, 3], dtype=I32)


def test_a_batch_is_written_in_place():
    b = batch()
    at = b._desc.lens
    b.lens += 1
    b.lens.add_(1)
    b.lens[0] = 9
    assert b.lens.tolist() == [9, 7] and b.lens.data_ptr() == at == b._desc.lens


@pytest.mark.parametrize("fmt", [S.NVFP4, S.MXFP4])
@pytest.mark.parametrize("name", ["k_codes", "k_scales", "v_codes", "v_scales", "texp"])
def test_a_cache_keeps_its_buffers(fmt, name):
    c = S.KVCache.empty(fmt, 2, 16, 1, 64, "cpu")
    old = getattr(c, name)
    with pytest.raises(AttributeError, match=name):
        setattr(c, name, torch.zeros(2, dtype=I32) if old is None else old.clone())
    assert getattr(c, name) is old
    if isinstance(old, torch.Tensor):
        c.__setattr__(name, old)
        old.fill_(1)
