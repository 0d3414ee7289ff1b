"""Plain references of the operators of a drafted step, in numpy with 64-bit arithmetic;
used by the tests only."""
from __future__ import annotations

import numpy as np

from serving_ref import EPS32, EPS_BF16, attention_tolerance


def rotate_ref(x, positions, turns, factor, interleaved):
    """x float64 [tokens, heads, D]; turns a position [dims / 2] in float64."""
    t = np.asarray(positions, np.float64)[:, None] * turns
    t = 2 * np.pi * (t - np.rint(t))
    c, s = (factor * f(t)[:, None] for f in (np.cos, np.sin))
    r = 2 * len(turns)
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    out = x.copy()
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def rotate_tolerance(x, ref, turns, factor, interleaved, bf16):
    """The fraction of a turn is rounded to fp32 (of at most half a turn: the angle by pi 2^-24), the
    library's sine and cosine are within 4 2^-24 (2 units), the factor and its products round
    by 2^-24 each, the two products of an element and their sum by 2^-24 each, all relative to
    (|a| + |b|) factor: pi + 4 + 2 + 3 < 13 times 2^-24.  Then one rounding to the type."""
    r = 2 * len(turns)
    a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    size = np.zeros_like(x)
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    err = 13 * EPS32 * abs(factor) * size
    return err + (EPS_BF16 * (np.abs(ref) + err) if bf16 else EPS32 * np.abs(ref))


def ancestors(parents):
    """Bool [n, n]: which rows each row of a tree sees (itself and its ancestors)."""
    n = len(parents)
    out = np.zeros((n, n), bool)
    for i in range(n):
        c = i
        while True:
            out[i, c] = True
            p = parents[c]
            if not 0 <= p < c:
                break
            c = p
    return out


def mask_words(sees, words):
    """Bool [rows, n] -> int32 [rows, words]."""
    rows, n = sees.shape
    bits = np.zeros((rows, words * 32), np.uint32)
    k = min(n, words * 32)
    bits[:, :k] = sees[:, :k]
    w = np.bitwise_or.reduce(bits.reshape(rows, words, 32) << np.arange(32, dtype=np.uint32), axis=-1)
    return w.astype(np.uint32).view(np.int32)


def tree_ref(q, kv, batch, q_heads, scale, sees):
    """fp64 attention with sees[b] bool [new, new] in place of causality.  Returns out, W = sum p |v| / sum
    p, delta = max |scale| sum |q k|, floor = |scale| sum |q| max |k| and top = max |v|, over what each
    row sees."""
    T, _, D = q.shape
    out, W, top = (np.zeros((T, q_heads, D)) for _ in range(3))
    delta, floor = np.zeros((T, q_heads)), np.zeros((T, q_heads))
    for b, new in enumerate(batch.news):
        k, v = kv[b]
        n = int(batch.lens[b])
        context = n - new
        per = q_heads // k.shape[1] if n > 0 else 1
        for i in range(new):
            t = int(batch.starts[b]) + i
            seen = [p for p in range(n) if p < context or sees[b][i, p - context]]
            if not seen:
                continue
            for h in range(q_heads):
                kk, vv = k[seen, h // per], v[seen, h // per]
                s = scale * (kk @ q[t, h])
                p = np.exp(s - s.max())
                out[t, h] = p @ vv / p.sum()
                W[t, h] = p @ np.abs(vv) / p.sum()
                top[t, h] = np.abs(vv).max()
                delta[t, h] = abs(scale) * (np.abs(kk) @ np.abs(q[t, h])).max()
                floor[t, h] = abs(scale) * np.abs(q[t, h]).sum() * np.abs(kk).max()
    return out, W, delta, floor, top


def tree_tolerance(ref, W, delta, floor, top, D, n):
    """Keys and values are rounded as by the attention of many new tokens (attention_tolerance's
    prompt terms, with the largest value that the row sees): a scale to fp16 and its product with
    the code again.  Both are measured against the largest scale of the position (keys) or of the group so far
    (values): an element far below it is off by at most half of fp16's smallest step, 2^-25,
    of keys whose largest element is at least 7 2^-9, so 2^-18 of it: a logit by 2^-18 floor, a
    weight by twice that to first order (doubled for numerator and sum)."""
    tol = attention_tolerance(ref, W, delta, D, n, top, prompt=True)
    return tol + W * (4 * 2.0 ** -18 * floor)[..., None]


def verify_ref(probs, ids, parents, starts, u, draft=None):
    """The rule, a sequence at a time, in float64: (path, accepted, next)."""
    T, V = probs.shape
    path = np.full(T, -1, np.int32)
    accepted, drawn = [], []
    for b in range(len(starts) - 1):
        f, n = int(starts[b]), int(starts[b + 1] - starts[b])
        if n == 0:
            accepted.append(0)
            drawn.append(-1)
            continue
        cur, at = 0, 1
        path[f] = 0
        while True:
            p = probs[f + cur].astype(np.float64)
            whole = p.copy()
            rest, went = 1.0, None
            for c in range(cur + 1, n):
                if parents[f + c] != cur:
                    continue
                tok = int(ids[f + c])
                inside = 0 <= tok < V
                pc = p[tok] if inside else 0.0
                if draft is not None:
                    qc = float(draft[f + cur, tok]) if inside else 0.0
                    if float(u[f + c]) * qc < pc:
                        went = c
                    else:
                        p = np.maximum(p - draft[f + cur].astype(np.float64), 0)
                    break
                if float(u[f + c]) * rest < pc:
                    went = c
                    break
                rest -= pc
                if inside:
                    p[tok] = 0.0
            if went is None:
                break
            cur = went
            path[f + at] = cur
            at += 1
        accepted.append(at)
        if not p.sum() > 0:
            p = whole
        upto = np.cumsum(p)
        passed = np.flatnonzero((upto > float(u[f]) * upto[-1]) & (p > 0))
        some = np.flatnonzero(p > 0)
        drawn.append(int(passed[0]) if passed.size else (int(some[-1]) if some.size else -1))
    return path, np.array(accepted, np.int32), np.array(drawn, np.int32)


def random_tree(g, n, reach=4):
    """Parents of n rows, each an earlier row."""
    return [-1] + [int(g.integers(max(0, i - 1 - reach), i)) for i in range(1, n)]
