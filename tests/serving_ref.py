"""Plain references of the int8 activation and 4-bit cache operators, in numpy
with 64-bit arithmetic and the oracle's quantizers; used by the tests only."""
from __future__ import annotations

import numpy as np

import oracle
import workload

EPS32 = 2.0 ** -24  # half a step of fp32, relative
EPS_BF16 = 2.0 ** -8
EPS_F16 = 2.0 ** -11


def tokens_ref(x):
    """(codes int8 [M, K], scales float32 [M], sums int32 [M]) by the oracle's 8-bit rule."""
    _, scales, q = oracle.quantize_pack(x, 8)
    q = np.asarray(q)
    return q.astype(np.int8), scales, q.sum(axis=1).astype(np.int32)


def pad128(codes):
    M, K = codes.shape
    out = np.zeros((M, -(-K // 128) * 128), np.int8)
    out[:, :K] = codes
    return out


def product_ref(codes, x_scales, q, w_scales):
    """Exact integer product (fp64 holds every partial sum) times the two scales in fp64;
    q: int codes less their zero point."""
    acc = codes.astype(np.float64) @ q.astype(np.float64).T
    return acc * x_scales.astype(np.float64)[:, None] * w_scales.astype(np.float64)[None, :]


def key_order(D):
    """Storage place of each dimension of a key row (codes of 4 bits, from the low bits up)."""
    d = np.arange(D)
    return (((d % 32) // 8) * (D // 32) + d // 32) * 8 + d % 8


def value_order(D):
    d = np.arange(D)
    return (d % 16) * (D // 16) + d // 16


def words(codes, order):
    """Codes -8 .. 7 [..., D] -> uint32 words [..., D / 8] in storage order."""
    u = np.zeros(codes.shape, np.uint32)
    u[..., order] = (codes + 8).astype(np.uint32)
    u = u.reshape(*codes.shape[:-1], codes.shape[-1] // 8, 8)
    return np.bitwise_or.reduce(u << np.arange(0, 32, 4, dtype=np.uint32), axis=-1)


def codes_of(w, order):
    """The inverse of ``words``: int codes [..., D]."""
    u = (w.astype(np.uint32)[..., None] >> np.arange(0, 32, 4, dtype=np.uint32)) & 15
    u = u.reshape(*w.shape[:-1], w.shape[-1] * 8)
    return u[..., order].astype(np.int64) - 8


def group4(x, g):
    """The oracle's 4-bit group quantizer over the last axis: (codes, scales [..., D / g])."""
    D = x.shape[-1]
    flat = np.ascontiguousarray(x.reshape(-1, D))
    _, scales, q = oracle.quantize_pack_group(flat, 4, g)
    return (np.asarray(q).reshape(x.shape).astype(np.int64),
            np.asarray(scales).reshape(*x.shape[:-1], D // g))


def values(codes, scales, g):
    """fl32(q * s) as float32 [..., D]."""
    return codes.astype(np.float32) * np.repeat(scales, g, axis=-1)


class Batch:
    """Random sequences over a page pool: lens, new tokens, a scattered page table."""

    def __init__(self, seed, lens, news, page, extra_pages=2, width=None, pad=0):
        g = np.random.default_rng(seed)
        self.page = page
        self.lens = np.asarray(lens, np.int32)
        self.news = list(news)
        self.starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.tokens = int(self.starts[-1])
        per = [-(-max(int(n), 0) // page) for n in lens]
        self.pages = sum(per) + extra_pages
        order = g.permutation(self.pages)
        self.width = max(max(per), 1) if width is None else width
        self.table = np.full((len(per), self.width), pad, np.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n

    def places(self, b, n):
        """(pages, offsets) of the first n positions of sequence b."""
        p = np.arange(n)
        return self.table[b, p // self.page], p % self.page


def attention_ref(q, kv, batch, q_heads, scale):
    """fp64 attention and the pieces of its error bound.  q float64 [T, Hq, D]; kv: list of
    (k, v) float64 [len, Hkv, D] per sequence.  Returns (out, W, delta): W[t,h,d] = sum p |v|
    / sum p, delta[t,h] = max over positions of scale * sum |q k|."""
    T, _, D = q.shape
    out = np.zeros((T, q_heads, D))
    W = np.zeros_like(out)
    delta = np.zeros((T, q_heads))
    for b, n_new in enumerate(batch.news):
        k, v = kv[b]
        n = int(batch.lens[b])
        per = q_heads // k.shape[1] if n > 0 else 1
        for i in range(n_new):
            t = int(batch.starts[b]) + i
            seen = n - n_new + i + 1
            if seen <= 0:
                continue
            for h in range(q_heads):
                kk, vv = k[:seen, h // per], v[:seen, h // per]
                s = scale * (kk @ q[t, h])
                p = np.exp(s - s.max())
                out[t, h] = p @ vv / p.sum()
                W[t, h] = p @ np.abs(vv) / p.sum()
                delta[t, h] = np.abs(scale) * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, W, delta


def attention_tolerance(ref, W, delta, D, n, v_max, prompt=False):
    """How far cache4_attention may be from attention_ref, from the roundings that it makes:
    * the output is rounded to bf16: 2^-8 |ref|;
    * a logit: D products are exact, their fp32 sum and the scalings round at most D + 8 times,
      each within 2^-24 of the sum of magnitudes (delta); the logit's maximum and exponent
      argument round again within that; an error e of a logit moves its weight by e (to first
      order, doubled here for the numerator and the sum it is divided by);
    * the hardware's exp2 is within 2^-22 of a weight;
    * weight times value scale rounds to fp32 (2^-24) and fp16 (2^-11), below fp16's normal range
      by 2^-25 of 2^14 of the largest scale: n * 2^-38 * v_max covers |code| <= 8;
    * n products and the weights' sum accumulate in fp32: 2 n 2^-24, with the rescalings.
    prompt: the kernel for many new tokens also rounds each scale to fp16 and its product with
    the code again, 2 * 2^-11 of a key (so of a logit's magnitudes) and of a value; a weight below
    fp16's normal range is off by 2^-25 of at least 2^6, a scale below it by 2^-25 of 2^10."""
    e = 2 * (D + 16) * EPS32 * delta[..., None]
    rel = EPS_F16 + 2 * (2.0 ** -22) + 4 * n * EPS32 + e
    if prompt:
        rel = rel + 2 * EPS_F16 + 2 * 2 * EPS_F16 * delta[..., None]
        v_max = v_max * (1 + 2.0 ** 7)  # n 2^-38 -> n 2^-31, which covers both
    return EPS_BF16 * np.abs(ref) * (1 + 2.0 ** -7) + W * rel * (1 + 2.0 ** -6) + n * 2.0 ** -38 * v_max


def bf16(a):
    return workload.bf16_from_f32(np.asarray(a, np.float32))


def widen(h):
    return workload.bf16_to_f32(h)
