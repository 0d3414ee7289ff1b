"""The int8 products at the ends of their scales' range: the exact sum times the two scales, wherever
that is a finite fp32 number."""
from __future__ import annotations

import numpy as np
import pytest

import mixed_precision_weight_dq_amd as dq
from gpu_util import report, torch
from serving_ref import EPS32, EPS_BF16, bf16, pad128, product_ref, tokens_ref, widen
from test_gpu_tokens_i8 import gpu_weights, weights_i8

pytestmark = pytest.mark.gpu

# M, N, K: the kernel of few tokens, of few tiles, of many
SHAPES = [(5, 70, 700), (40, 300, 700), (300, 12000, 260)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_scales_at_both_ends(shape, out):
    """x near the largest bf16 with small weight scales (the sum times the token's scale alone is past
    fp32), x near 2^-126 with large ones, and ordinary tokens among them.  A y that is subnormal may be
    off by half of fp32's smallest step more at each of the three roundings."""
    t = torch()
    M, N, K = shape
    bits = 6
    g = np.random.default_rng(M)
    x = g.standard_normal((M, K)).astype(np.float32)
    x = x / np.abs(x).max(axis=1, keepdims=True)
    mags = np.array([3.3e38, 2.0 ** 126, 1.0, 2.0 ** -120, 2.0 ** 104, 2.0 ** 96 * 127, 2.0 ** 90])
    x = widen(bf16((x * mags[np.arange(M) % len(mags), None]).astype(np.float32)))
    codes, xs, sums = tokens_ref(x)
    packed, scales, zeros, q = weights_i8(3, N, K, bits, True)
    for mul in (2.0 ** -30, 1.0, 2.0 ** 60):
        sw = (scales * np.float32(mul)).astype(np.float32)
        P, S, Z = gpu_weights(packed, sw, zeros)
        report("int8 product M=%d N=%d K=%d, scales x %g, %s" % (M, N, K, mul, out))
        y = dq.gemm_i8(t.from_numpy(pad128(codes)).cuda(), t.from_numpy(xs).cuda(),
                       t.from_numpy(sums).cuda(), P, S, K, bits, zeros=Z,
                       dtype=t.float32 if out == "f32" else t.bfloat16)
        t.cuda.synchronize()
        got = y.double().cpu().numpy()
        ref = product_ref(codes, xs, q, sw)
        tol = np.abs(ref) * (3 * EPS32 if out == "f32" else EPS_BF16 + 4 * EPS32) * (1 + 1e-6)
        tol += 3 * 2.0 ** -150 if out == "f32" else 2.0 ** -134
        top = float(t.finfo(t.float32 if out == "f32" else t.bfloat16).max)
        fits = np.abs(ref) < top * (1 - 2.0 ** -9)
        assert (np.abs(got - ref) <= tol)[fits].all()
        past = np.abs(ref) > top * (1 + 2.0 ** -7)
        assert (got == np.copysign(np.inf, ref))[past].all()
