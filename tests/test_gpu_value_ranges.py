"""Few new tokens over the 4-bit cache where the magnitudes of values lie far apart: what a row does
not see, and groups whose codes are all 0 (their stored scale is 1/7), must not cost the bits of
what it sees."""
from __future__ import annotations

import numpy as np
import pytest

from gpu_util import report
from serving_ref import Batch
from serving_ranges import FACTORS, GEOMETRY, check, prompt_batch, vectors, with_zeros

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,g", GEOMETRY)
def test_decode_small_values_beside_zero_groups(D, g):
    n, H, per = 150, 2, 4
    batch = Batch(1, [n, n], [1, 3], 16)
    for factor in FACTORS:
        k = vectors(1, 2 * n, H, D)
        v = with_zeros(vectors(2, 2 * n, H, D) * np.float32(factor), n, g)
        for hints in (None, dict(max_q=3, max_len=200000)):
            report("decode D=%d g=%d values x %g with zero groups %s" % (D, g, factor, hints))
            check(batch, H, per, D, g, k, v, False, hints=hints)


@pytest.mark.parametrize("D,g", GEOMETRY)
def test_draft_later_token_far_larger(D, g):
    """Five drafted tokens, the last ones' values far larger than any before: the rows before them do
    not see them."""
    H, per = 2, 2
    for n in (5, 20, 150, 133):
        batch = Batch(2, [n, 40], [5, 1], 16)
        for up in (2.0 ** 20, 2.0 ** 45, 2.0 ** 90, 2.0 ** 120):
            k, v = vectors(3, n + 40, H, D), vectors(4, n + 40, H, D)
            v[n - 1] *= np.float32(up)
            v[n - 2] *= np.float32(up ** 0.5)
            report("draft D=%d g=%d n=%d last x %g" % (D, g, n, up))
            check(batch, H, per, D, g, k, v, False)


@pytest.mark.parametrize("D,g", GEOMETRY)
def test_draft_magnitudes_and_zeros(D, g):
    """Every token's values of another magnitude, up to 2^60 either way, with zero groups and whole
    zero tokens among them."""
    H, per = 2, 3
    rng = np.random.default_rng(D + g)
    for batch in (Batch(5, [700, 40, 9], [6, 2, 9], 16), Batch(6, [60] * 70, [2] * 70, 32)):
        n = int(batch.lens.sum())
        k, v = vectors(18, n, H, D), vectors(19, n, H, D)
        v *= np.exp2(rng.integers(-60, 61, (n, 1, 1))).astype(np.float32)
        zero = rng.random((n, H, D // g)) < 0.3
        zero[::7] = True
        v[np.repeat(zero, g, axis=2)] = 0
        for hints in (None, dict(max_q=9, max_len=200000)):
            report("drafts D=%d g=%d magnitudes and zeros %s" % (D, g, hints))
            check(batch, H, per, D, g, k, v, False, hints=hints)


@pytest.mark.parametrize("D,g", GEOMETRY)
def test_decode_largest_values(D, g):
    """Values up to 2^124, whole and in parts that are joined."""
    H, per = 2, 4
    batch = Batch(3, [1500, 40], [1, 3], 16)
    many = Batch(4, [90] * 70, [1] * 70, 16)
    for hints in (None, dict(max_q=3, max_len=200000)):
        report("decode D=%d g=%d values of 2^121 %s" % (D, g, hints))
        for b in (batch, many):
            n = int(b.lens.sum())
            v = np.abs(vectors(17, n, H, D)) * np.float32(2.0 ** 121)
            check(b, H, per, D, g, vectors(16, n, H, D), v, False, scale=2.0 ** -9, hints=hints)


def test_few_rows_keep_exact_codes():
    """max_q that names few rows takes the kernel that multiplies the codes exactly, for a prompt too:
    its bound is the one of few new tokens."""
    D, g, n, H, per = 128, 32, 160, 4, 2
    batch = prompt_batch(7, n)
    k, v = vectors(14, 13 * n, H, D), vectors(15, 13 * n, H, D)
    for hints in (dict(max_q=1, max_len=n), dict(max_q=31, max_len=200000)):
        report("prompts by the kernel of few new tokens %s" % hints)
        check(batch, H, per, D, g, k, v, False, hints=hints)
