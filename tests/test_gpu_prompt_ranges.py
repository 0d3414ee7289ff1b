"""Prompts over the 4-bit cache, through the kernel of many new tokens, where the magnitudes of
values and keys lie far apart: what a row does not see, and groups whose codes are all 0 (their
stored scale is 1/7), must not cost the bits of what it sees."""
from __future__ import annotations

import numpy as np
import pytest

import mixed_precision_weight_dq_amd as dq
from gpu_util import bf16_gpu, report, torch
from serving_ref import Batch, bf16, widen
from serving_ranges import (FACTORS, GEOMETRY, check, gpu, prompt_batch, range_tolerance, reference,
                            vectors, with_zeros)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hints", [None, dict(max_q=160, max_len=200000), dict(max_q=160, max_len=1)])
@pytest.mark.parametrize("D,g", GEOMETRY)
def test_prompt_small_values_beside_zero_groups(D, g, hints):
    n, H, per = 160, 4, 2
    batch = prompt_batch(3, n)
    k = vectors(5, 13 * n, H, D)
    for factor in FACTORS:
        v = with_zeros(vectors(6, 13 * n, H, D) * np.float32(factor), n, g)
        report("prompts D=%d g=%d values x %g with zero groups %s" % (D, g, factor, hints))
        check(batch, H, per, D, g, k, v, True, hints=hints)


@pytest.mark.parametrize("D,g", GEOMETRY)
def test_prompt_later_token_far_larger(D, g):
    """In each sequence one token's values, somewhere, are far larger than the ones before."""
    n, H, per, count = 160, 4, 2, 13
    batch = prompt_batch(4, n)
    at = np.arange(count) * 12 + 3
    for up in (2.0 ** 20, 2.0 ** 50, 2.0 ** 90, 2.0 ** 120):
        k, v = vectors(7, count * n, H, D), vectors(8, count * n, H, D)
        v[np.arange(count) * n + at] *= np.float32(up)
        for hints in (None, dict(max_q=n, max_len=200000)):
            report("prompts D=%d g=%d one token x %g %s" % (D, g, up, hints))
            check(batch, H, per, D, g, k, v, True, hints=hints)


@pytest.mark.parametrize("D,g", GEOMETRY)
def test_prompt_largest_values(D, g):
    """Values up to 2^124, whole and in parts that are joined."""
    n, H, per, count = 150, 4, 2, 13
    k, v = vectors(16, count * n, H, D), vectors(17, count * n, H, D) * np.float32(2.0 ** 121)
    for hints in (None, dict(max_q=n, max_len=200000)):
        report("prompts D=%d g=%d values of 2^121 %s" % (D, g, hints))
        check(prompt_batch(8, n), H, per, D, g, k, v, True, hints=hints)


@pytest.mark.parametrize("D,g", GEOMETRY)
def test_prompt_magnitudes_and_zeros(D, g):
    """Every token's values of another magnitude, up to 2^60 either way, with zero groups and whole
    zero tokens among them."""
    n, H, per, count = 140, 4, 3, 13
    rng = np.random.default_rng(D + g)
    k, v = vectors(18, count * n, H, D), vectors(19, count * n, H, D)
    v *= np.exp2(rng.integers(-60, 61, (count * n, 1, 1))).astype(np.float32)
    zero = rng.random((count * n, H, D // g)) < 0.3
    zero[::7] = True
    v[np.repeat(zero, g, axis=2)] = 0
    for hints in (None, dict(max_q=n, max_len=200000)):
        report("prompts D=%d g=%d magnitudes and zeros %s" % (D, g, hints))
        check(prompt_batch(9, n), H, per, D, g, k, v, True, hints=hints)


@pytest.mark.parametrize("D,g", [(64, 32), (128, 32), (128, 64), (256, 64)])
def test_prompt_groups_far_apart(D, g):
    """The groups of a head 2^18 apart, and each token's magnitude another: the bound is the head's."""
    n, H, per, count = 150, 4, 2, 13
    batch = prompt_batch(5, n)
    rng = np.random.default_rng(9)
    k, v = vectors(9, count * n, H, D), vectors(10, count * n, H, D)
    v[..., :g] *= np.float32(2.0 ** -18)
    v *= np.exp2(rng.integers(-12, 13, (count * n, 1, 1))).astype(np.float32)
    report("prompts D=%d g=%d groups far apart" % (D, g))
    check(batch, H, per, D, g, k, v, True)


@pytest.mark.parametrize("D,g", [(64, 32), (128, 32), (128, 128), (256, 64)])
def test_prompt_keys_beside_larger_ones(D, g):
    """Small keys and large queries: keys that a row does not see, and zero groups and tokens of
    keys, do not cost the logits their bits."""
    n, H, per, count = 160, 4, 2, 13
    batch = prompt_batch(6, n)
    k, v = vectors(11, count * n, H, D), vectors(12, count * n, H, D)
    k = with_zeros(k * np.float32(2.0 ** -40), n, g)
    report("prompts D=%d g=%d keys x 2^-40 with zero groups" % (D, g))
    check(batch, H, per, D, g, k, v, True, q_mul=2.0 ** 40)
    at = np.arange(count) * 12 + 3
    k = vectors(13, count * n, H, D)
    k[np.arange(count) * n + at] *= np.float32(2.0 ** 35)
    report("prompts D=%d g=%d one key x 2^35" % (D, g))
    check_before(batch, H, per, D, g, k, v, at)


def check_before(batch, H, per, D, g, k, v, at):
    """As check, for the rows before position at[b] of each sequence b alone: the cache holds all of
    them, the reference is computed on a batch that ends there."""
    t = torch()
    n, count = int(batch.lens[0]), len(batch.lens)
    full = gpu(batch.starts)
    cache = dq.Cache4.empty(batch.pages, H, D, batch.page, g)
    dq.cache4_append(cache, gpu(k), gpu(v), full, gpu(batch.lens), gpu(batch.table))
    kd, vd = dq.cache4_read(cache, count * n, full, gpu(batch.lens), gpu(batch.table))
    qb = bf16(np.random.default_rng(1).standard_normal((count * n, H * per, D)))
    out = dq.cache4_attention(cache, bf16_gpu(qb), full, gpu(batch.lens), gpu(batch.table), max_q=n, max_len=n)
    t.cuda.synchronize()
    rows = np.concatenate([b * n + np.arange(a) for b, a in enumerate(at)])
    short = Batch(0, list(at), list(at), batch.page)
    kv = [(kd[b * n:b * n + a].double().cpu().numpy(), vd[b * n:b * n + a].double().cpu().numpy())
          for b, a in enumerate(at)]
    ref, W, delta, top = reference(widen(qb)[rows].astype(np.float64), kv, short, H * per, D ** -0.5)
    tol = range_tolerance(ref, W, delta, top, D, n, True)
    got = out.double().cpu().numpy()[rows]
    assert (np.abs(got - ref) <= tol).all()
