"""Refusals of the int8 activation and 4-bit cache entry points: every invalid argument is
returned on the host before any HIP call, so these run without a GPU (the fake device
addresses are never dereferenced), and the torch layer's own checks."""
from __future__ import annotations

import ctypes

import pytest

import mixed_precision_weight_dq_amd as dq

A = 1 << 20
MIS = A + 4


def test_token_row_bytes():
    for K in (1, 127, 128, 129, 4096, 5121, 65536):
        assert dq.dq_token_row_bytes(K) == -(-K // 128) * 128
    for K in (0, -1, 65537):
        assert dq.dq_token_row_bytes(K) == 0


def test_quantize_tokens_refusals():
    ok = dict(x=A, x_dtype=dq.DQ_BF16, M=4, K=64, codes=A, scales=A, sums=A)
    call = lambda **kw: dq.dq_quantize_tokens(**{**ok, **kw})
    for name in ("x", "codes", "scales", "sums"):
        assert call(**{name: 0}) == dq.DQ_ERR_NULL
    for M, K in ((0, 64), (1 << 31, 64), (4, 0), (4, 65537)):
        assert call(M=M, K=K) == dq.DQ_ERR_SHAPE
    assert call(x_dtype=2) == dq.DQ_ERR_DTYPE
    assert call(x=MIS) == call(codes=MIS) == call(scales=A + 2) == call(sums=A + 1) == dq.DQ_ERR_ALIGN


@pytest.mark.parametrize("name", ["dq_gemv_i8", "dq_gemm_i8"])
def test_product_refusals(name):
    ok = dict(x=A, x_scales=A, x_sums=A, M=4, packed=A, scales=A, zeros=0, N=8, K=64, bits=4, y=A,
              y_dtype=dq.DQ_F32)
    call = lambda **kw: getattr(dq, name)(**{**ok, **kw})
    for arg in ("x", "x_scales", "x_sums", "packed", "scales", "y"):
        assert call(**{arg: 0}) == dq.DQ_ERR_NULL
    for bits in (0, 1, 9, 15, 16):
        assert call(bits=bits) == dq.DQ_ERR_BITS
    for kw in (dict(M=0), dict(N=0), dict(K=0), dict(K=65537), dict(N=1 << 31), dict(M=1 << 31)):
        assert call(**kw) == dq.DQ_ERR_SHAPE
    if name == "dq_gemv_i8":
        assert call(M=17) == dq.DQ_ERR_SHAPE
    assert call(y_dtype=3) == dq.DQ_ERR_DTYPE
    for kw in (dict(x=MIS), dict(packed=MIS), dict(scales=A + 2), dict(x_scales=A + 1),
               dict(x_sums=A + 2), dict(zeros=A + 2), dict(y=A + 2)):
        assert call(**kw) == dq.DQ_ERR_ALIGN
    assert call(y=A + 1, y_dtype=dq.DQ_BF16) == dq.DQ_ERR_ALIGN


CACHE = dict(k_codes=A, v_codes=A, k_scales=A, v_scales=A, pages=4, kv_heads=2, head_dim=64,
             page_size=16, group=32)
BATCH = dict(starts=A, lens=A, table=A, table_width=2, count=3)


def structs(kw):
    cache = dq.DQCache4(**{k: kw.pop(k, v) for k, v in CACHE.items()})
    batch = dq.DQCache4Batch(**{k: kw.pop(k, v) for k, v in BATCH.items()})
    return cache, batch


def append(**kw):
    c, b = structs(kw)
    return dq.dq_cache4_append(c, b, **{**dict(k=A, v=A, dtype=dq.DQ_BF16, tokens=3, k_stride=128,
                                               v_stride=128), **kw})


def read(**kw):
    c, b = structs(kw)
    return dq.dq_cache4_read(c, b, **{**dict(k=A, v=A, dtype=dq.DQ_BF16, tokens=3), **kw})


def attend(**kw):
    c, b = structs(kw)
    return dq.dq_cache4_attention(c, b, **{**dict(q=A, tokens=3, q_stride=256, q_heads=4, scale=0.1,
                                                  max_q=1, max_len=30, out=A, workspace=A,
                                                  workspace_bytes=1 << 40), **kw})


@pytest.mark.parametrize("call", [append, read, attend])
def test_cache4_refusals(call):
    for name in ("k_codes", "v_codes", "k_scales", "v_scales", "starts", "lens", "table"):
        assert call(**{name: 0}) == dq.DQ_ERR_NULL
        assert call(**{name: A + (2 if name in BATCH else 4)}) == dq.DQ_ERR_ALIGN
    for kw in (dict(head_dim=32), dict(head_dim=96), dict(head_dim=512), dict(page_size=8),
               dict(page_size=48), dict(page_size=512), dict(group=16), dict(group=128), dict(group=0),
               dict(kv_heads=0), dict(kv_heads=1025), dict(pages=0), dict(pages=1 << 31),
               dict(count=0), dict(count=65536), dict(table_width=0), dict(table_width=(1 << 24) + 1),
               dict(tokens=0), dict(tokens=1 << 31)):
        assert call(**kw) == dq.DQ_ERR_SHAPE, kw


def test_append_and_read_refusals():
    for call in (append, read):
        assert call(k=0) == call(v=0) == dq.DQ_ERR_NULL
        assert call(k=MIS) == call(v=MIS) == dq.DQ_ERR_ALIGN
        assert call(dtype=2) == call(dtype=-1) == dq.DQ_ERR_DTYPE
    for kw in (dict(k_stride=127), dict(v_stride=120), dict(k_stride=132), dict(v_stride=-128),
               dict(k_stride=(1 << 32) + 8)):
        assert append(**kw) == dq.DQ_ERR_SHAPE


def test_attention_refusals():
    assert attend(q=0) == attend(out=0) == dq.DQ_ERR_NULL
    assert attend(q=MIS) == attend(out=MIS) == attend(workspace=MIS) == dq.DQ_ERR_ALIGN
    for kw in (dict(q_heads=0), dict(q_heads=3), dict(q_heads=1026), dict(q_stride=255),
               dict(q_stride=260), dict(max_q=0), dict(max_len=0)):
        assert attend(**kw) == dq.DQ_ERR_SHAPE, kw
    for scale in (float("inf"), float("nan")):
        assert attend(scale=scale) == dq.DQ_ERR_VALUE


def test_attention_workspace():
    """The size is 0 for refused arguments, never less for a longer cache, and checked."""
    c, _ = structs({})
    size = lambda **kw: dq.dq_cache4_attention_workspace(
        c, **{**dict(count=2, tokens=2, q_heads=4, max_q=1, max_len=100), **kw})
    for kw in (dict(count=0), dict(tokens=0), dict(q_heads=3), dict(max_q=0), dict(max_len=0)):
        assert size(**kw) == 0
    long = size(max_len=1 << 17)
    assert long >= size() >= 0
    if long:
        kw = dict(count=2, tokens=2, max_len=1 << 17)
        assert attend(workspace=0, **kw) == dq.DQ_ERR_NULL
        assert attend(workspace_bytes=long - 1, **kw) == dq.DQ_ERR_SHAPE


def test_torch_layer_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        dq.quantize_tokens(x)
    codes = torch.zeros(2, 128, dtype=torch.int8)
    with pytest.raises(ValueError):
        dq.gemv_i8(codes, torch.zeros(2), torch.zeros(2, dtype=torch.int32),
                   torch.zeros(3, 32, dtype=torch.int32), torch.zeros(3), 64, 4)
    w, s = torch.zeros(1, 1, 16, 8, dtype=torch.int32), torch.zeros(1, 1, 2, 16)
    with pytest.raises(ValueError):
        dq.Cache4(w, w, s, s)
    with pytest.raises(dq.DQError):
        dq.Cache4.empty(1, 1, 80, device="cpu")
    with pytest.raises(TypeError):
        dq.quantize_tokens([1.0])
