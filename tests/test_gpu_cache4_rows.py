"""Attention over the 4-bit cache: which rows become NaN."""
from __future__ import annotations

import numpy as np
import pytest

import mixed_precision_weight_dq_amd as dq
from gpu_util import bf16_gpu, report, torch
from serving_ref import Batch, bf16
from serving_ranges import gpu, vectors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,g", [(64, 32), (128, 32), (256, 128)])
@pytest.mark.parametrize("news,hints", [(12, dict(max_q=12, max_len=64)), (12, dict(max_q=12, max_len=200000)),
                                        (150, dict(max_q=150, max_len=200)), (150, dict(max_q=150, max_len=200000))])
def test_length_past_the_table(D, g, news, hints):
    """Tokens on both sides of the table's end: those that see only held positions are what they are
    in a call that ends there, the ones behind it NaN; the sequences beside it as ever."""
    t = torch()
    H, per, page, count = 4, 2, 16, 13
    width = 10
    held = width * page
    past = 5 if news < 100 else 37  # cached tokens past the table
    lens = np.array([held + past] + [held - 7 * b for b in range(1, count)], np.int32)
    starts = (np.arange(count + 1) * news).astype(np.int32)
    table = np.arange(count * width, dtype=np.int32).reshape(count, width)
    cache = dq.Cache4.empty(count * width, H, D, page, g)
    k, v = vectors(1, count * held, H, D), vectors(2, count * held, H, D)
    full = gpu((np.arange(count + 1) * held).astype(np.int32))
    dq.cache4_append(cache, gpu(k), gpu(v), full, gpu(np.full(count, held, np.int32)), gpu(table))
    q = bf16_gpu(bf16(np.random.default_rng(3).standard_normal((count * news, H * per, D))))
    report("attention D=%d g=%d, %d of %d tokens past the table %s" % (D, g, past, news, hints))
    out = dq.cache4_attention(cache, q, gpu(starts), gpu(lens), gpu(table), **hints)
    t.cuda.synchronize()
    inside = news - past
    assert bool(t.isnan(out[inside:news]).all())
    assert bool(t.isfinite(out[:inside]).all()) and bool(t.isfinite(out[news:]).all())
    # the same tokens in a call whose first sequence ends at the table's end; the rows lie in other
    # tiles and stretches there, so they agree within the roundings of both: 2^-8 each to bf16, and
    # a weight's 2^-11 (keys and values rounded too in the kernel of many rows) of sum p |v| / sum p,
    # below the largest value, whose logits are below 2^5
    lens[0] = held
    starts[1:] -= past
    near = dq.cache4_attention(cache, t.cat([q[:inside], q[news:]]).contiguous(), gpu(starts), gpu(lens),
                               gpu(table), **hints).float()
    far = t.cat([out[:inside], out[news:]]).float()
    top = float(np.abs(v).max())
    assert bool(((far - near).abs() <= 2.0 ** -7 * near.abs() + 2.0 ** -4 * top).all())


@pytest.mark.parametrize("D,g", [(64, 32), (128, 32), (256, 32)])
@pytest.mark.parametrize("hints", [dict(max_q=1, max_len=300), dict(max_q=1, max_len=200000),
                                   dict(max_q=160, max_len=300)])
def test_nan_values_of_vanishing_weight(D, g, hints):
    """A value group with a NaN makes its dimensions NaN in every row that sees it, however small the
    weight: here below 2^-500, which is 0 in fp32."""
    t = torch()
    n, H, per, count = 160, 4, 2, 13
    batch = Batch(1, [n] * count, [n] * count, 16)
    k, v = vectors(3, count * n, H, D), vectors(4, count * n, H, D)
    at = 70
    k[2 * n + at] = -40.0  # of the queries, all positive: a logit far below the others
    v[2 * n + at, 1, g + 3] = np.nan
    cache = dq.Cache4.empty(batch.pages, H, D, 16, g)
    m = gpu(batch.starts), gpu(batch.lens), gpu(batch.table)
    dq.cache4_append(cache, gpu(k), gpu(v), *m)
    q = bf16_gpu(bf16(np.abs(np.random.default_rng(5).standard_normal((count * n, H * per, D))) + 2.0))
    report("attention D=%d g=%d, a NaN of vanishing weight %s" % (D, g, hints))
    out = dq.cache4_attention(cache, q, *m, **hints)
    t.cuda.synchronize()
    nan = np.zeros(out.shape, bool)
    nan[2 * n + at:3 * n, per:2 * per, g:2 * g] = True
    assert np.array_equal(t.isnan(out).cpu().numpy(), nan)
