"""Attention over the 4-bit cache: which rows become NaN."""
from __future__ import annotations

import numpy as np
import pytest

import mixed_precision_weight_dq_amd as dq
from gpu_util import bf16_gpu, report, torch
from serving_ref import Batch, bf16
from serving_ranges import gpu, vectors

pytestmark = pytest.mark.gpu


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
