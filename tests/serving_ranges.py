"""What the tests of the cache's ranges share: inputs whose magnitudes differ along a sequence,
and a bound that is relative to what each row may see."""
from __future__ import annotations

import numpy as np

import mixed_precision_weight_dq_amd as dq
from gpu_util import bf16_gpu, torch
from serving_ref import Batch, attention_tolerance, bf16, widen

GEOMETRY = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]
FACTORS = [1e-5, 1e-9, 1e-13, 1e-25]


def gpu(a):
    return torch().from_numpy(np.ascontiguousarray(a)).cuda()


def vectors(seed, n, H, D):
    return np.random.default_rng(seed).standard_normal((n, H, D)).astype(np.float32)


def with_zeros(x, n, g):
    """An all-zero token, an all-zero group of another, in every sequence of n tokens."""
    x = x.reshape(-1, n, *x.shape[1:])
    x[:, n // 3] = 0
    x[:, n // 2, :, :g] = 0
    x[:, 5, :, -g:] = 0
    return x.reshape(-1, *x.shape[2:])


def reference(q, kv, batch, q_heads, scale):
    """serving_ref.attention_ref's (out, W, delta), a sequence's head at a time, and the largest |v| of
    the positions and the kv head that a row sees, [tokens, q_heads, 1]."""
    T, _, D = q.shape
    out, W = np.zeros((T, q_heads, D)), np.zeros((T, q_heads, D))
    delta, top = np.zeros((T, q_heads)), np.zeros((T, q_heads, 1))
    for b, new in enumerate(batch.news):
        k, v = kv[b]
        n, first = int(batch.lens[b]), int(batch.starts[b])
        seen = n - new + 1 + np.arange(new)
        rows = np.flatnonzero(seen > 0)
        if not rows.size:
            continue
        at, seen = first + rows, seen[rows]
        hidden = np.arange(n)[None] >= seen[:, None]
        largest = np.maximum.accumulate(np.abs(v).max(axis=-1), axis=0)
        for h in range(q_heads):
            kk, vv = k[:, h // (q_heads // k.shape[1])], v[:, h // (q_heads // k.shape[1])]
            s = np.where(hidden, -np.inf, scale * (q[at, h] @ kk.T))
            p = np.exp(s - s.max(axis=1, keepdims=True))
            p /= p.sum(axis=1, keepdims=True)
            out[at, h], W[at, h] = p @ vv, p @ np.abs(vv)
            delta[at, h] = abs(scale) * np.where(hidden, 0, np.abs(q[at, h]) @ np.abs(kk).T).max(axis=1)
            top[at, h, 0] = largest[seen - 1, h // (q_heads // k.shape[1])]
    return out, W, delta, top


def range_tolerance(ref, W, delta, top, D, n, prompt):
    """serving_ref.attention_tolerance with the largest value that each row sees (top) in place of the
    whole cache's.

    A weight (times its value's scale) below fp16's normal range is off by half of its smallest
    step, 2^-25.  Few new tokens: that is 2^-25 of 2^14 of the largest scale seen, times |code| <= 8
    of at least 7 such codes: n 2^-38 v, attention_tolerance's own term.  Many (prompt): a weight's
    reference is at least 2^6, a value in fp16 at most 2^14, and the largest value seen at least 7 *
    2^3, the exponents being multiples of 8: 2^-25 2^14 / (2^6 7 2^3) < 2^-22, which is 2^9 times the
    n 2^-38 (1 + 2^7) that attention_tolerance has for them."""
    return attention_tolerance(ref, W, delta, D, n, top * 2.0 ** 9 if prompt else top, prompt)


def check(batch, H, per, D, g, k, v, prompt, scale=None, q_mul=1.0, seed=3, hints=None):
    """Appends k, v (all cached tokens of all sequences) and attends, against fp64 on what the cache
    holds; returns nothing, fails with the first row that is off."""
    t = torch()
    T = int(batch.lens.sum())
    full = gpu(np.concatenate([[0], np.cumsum(batch.lens)]).astype(np.int32))
    lens, table, starts = gpu(batch.lens), gpu(batch.table), gpu(batch.starts)
    cache = dq.Cache4.empty(batch.pages, H, D, batch.page, g)
    dq.cache4_append(cache, gpu(k), gpu(v), full, lens, table)
    kd, vd = dq.cache4_read(cache, T, full, lens, table)
    cuts = np.cumsum(batch.lens)[:-1]
    kv = list(zip(np.split(kd.double().cpu().numpy(), cuts), np.split(vd.double().cpu().numpy(), cuts)))
    qb = bf16(np.random.default_rng(seed).standard_normal((batch.tokens, H * per, D)) * q_mul)
    hints = hints or dict(max_q=max(batch.news), max_len=int(batch.lens.max()))
    out = dq.cache4_attention(cache, bf16_gpu(qb), starts, lens, table, scale=scale, **hints)
    t.cuda.synchronize()
    got = out.double().cpu().numpy()
    ref, W, delta, top = reference(widen(qb).astype(np.float64), kv, batch, H * per,
                                   D ** -0.5 if scale is None else scale)
    tol = range_tolerance(ref, W, delta, top, D, int(batch.lens.max()), prompt)
    bad = ~(np.abs(got - ref) <= tol)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        rows = np.unique(np.argwhere(bad)[:, 0])
        raise AssertionError("%d of %d off in %d rows, first %s: %r ref %r tol %r" % (
            bad.sum(), bad.size, rows.size, at, got[at], ref[at], tol[at]))


def prompt_batch(seed, n, page=16, count=13):
    """First prompts of n tokens: with 4 kv heads of 2 query heads and n > 128, units enough for the
    kernel of many new tokens."""
    return Batch(seed, [n] * count, [n] * count, page)
