"""A Cache4 keeps the addresses of its tensors: it cannot be made to use old ones.  The tensors here
stand in for GPU tensors with addresses that nothing dereferences, so this runs without a GPU."""
from __future__ import annotations

import pytest

import mixed_precision_weight_dq_amd as dq


class Stand:
    """A contiguous tensor on GPU 0, as far as the argument checks look."""
    is_cuda = True
    device = "cuda:0"

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.at = dtype, shape, 1 << 20

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return self.at

    def stride(self):
        out, n = [], 1
        for s in reversed(self.shape):
            out.insert(0, n)
            n *= s
        return tuple(out)


def tensors(pages=4):
    torch = pytest.importorskip("torch")
    codes = [Stand(torch.int32, pages, 2, 16, 8) for _ in range(2)]
    scales = [Stand(torch.float32, pages, 2, 2, 16) for _ in range(2)]
    return codes + scales


def test_attributes_are_fixed():
    cache = dq.Cache4(*tensors())
    for name in ("k_codes", "v_codes", "k_scales", "v_scales", "pages", "kv_heads", "page_size",
                 "head_dim", "group", "device_index", "_c", "anything"):
        with pytest.raises(AttributeError):
            setattr(cache, name, 1)
    with pytest.raises(AttributeError):
        del cache.k_codes
    assert (cache.pages, cache.kv_heads, cache.page_size, cache.head_dim, cache.group) == (4, 2, 16, 64, 32)
    assert cache._struct().k_codes == 1 << 20


@pytest.mark.parametrize("which", range(4))
def test_moved_tensors_are_refused(which):
    torch = pytest.importorskip("torch")
    parts = tensors()
    cache = dq.Cache4(*parts)
    parts[which].at = 1 << 21  # as resize_ or an assignment to .data moves a tensor
    kv = Stand(torch.bfloat16, 3, 2, 64)
    meta = Stand(torch.int32, 2), Stand(torch.int32, 1), Stand(torch.int32, 1, 4)
    with pytest.raises(ValueError, match="moved"):
        dq.cache4_append(cache, kv, kv, *meta)
    with pytest.raises(ValueError, match="moved"):
        dq.cache4_read(cache, 3, *meta, k=Stand(torch.float32, 3, 2, 64), v=Stand(torch.float32, 3, 2, 64))
    with pytest.raises(ValueError, match="moved"):
        dq.cache4_attention(cache, kv, *meta, out=Stand(torch.bfloat16, 3, 2, 64))
