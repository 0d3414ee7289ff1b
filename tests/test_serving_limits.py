"""Serving operators at the ends of their arguments' ranges, without a GPU."""
from __future__ import annotations

import ctypes

import pytest

import mixed_precision_weight_dq_amd as dq

BIG = 2 ** 31 - 1
LIMIT = 2 * 512 * 128 * (4 * 128 + 8)  # the most that heads of 128 need: 512 workgroups of 128 rows


def cache(heads, D=128, g=32):
    p = ctypes.c_void_p(4096)
    return dq.DQCache4(p, p, p, p, BIG, heads, D, 16, g)


@pytest.mark.parametrize("heads,q_heads", [(1, 1), (1, 1024), (8, 64), (1024, 1024)])
@pytest.mark.parametrize("count", [1, 65535])
@pytest.mark.parametrize("max_q", [1, 1000, 2 ** 20, BIG, 2 ** 62])
@pytest.mark.parametrize("max_len", [1, 10 ** 6, BIG, 2 ** 62])
def test_workspace_bounds(heads, q_heads, count, max_q, max_len):
    """No product of sizes wraps: the workspace stays what its workgroups need."""
    need = dq.dq_cache4_attention_workspace(cache(heads), count, BIG, q_heads, max_q, max_len)
    assert 0 <= need <= LIMIT
    if count * heads == 1 and max_q == 1 and q_heads == 1 and max_len >= 10 ** 6:
        assert need == 512 * 2 * 16 * (4 * 128 + 8)


@pytest.mark.parametrize("scale", [3e38, -3e38, float("inf"), float("nan")])
def test_scale_refused(scale):
    p = ctypes.c_void_p(4096)
    batch = dq.DQCache4Batch(p, p, p, 4, 1)
    status = dq.load().dq_cache4_attention(cache(1), batch, p, 1, 128, 1, scale, 1, 64, p, p, 1 << 30, None)
    assert status == dq.DQ_ERR_VALUE
