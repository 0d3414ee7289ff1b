"""Int8 activations on the GPU: per-token codes, scales and sums bit for bit against the
oracle's 8-bit quantizer; integer products against an exact int64 product, within the three
fp32 roundings (and the one to bf16) that an output goes through.

Source: "量化" tutorial (aiknowledge.cn), "how quantization works", with one token as the
channel of x."""
from __future__ import annotations

import numpy as np
import pytest

import mixed_precision_weight_dq_amd as dq
import oracle
import workload
from gpu_util import bf16_gpu, f32_bits, report, torch, weights_gpu
from serving_ref import EPS32, EPS_BF16, pad128, product_ref, tokens_ref

pytestmark = pytest.mark.gpu

K_EDGES = [1, 7, 8, 31, 33, 127, 128, 129, 257, 1000, 2048, 4096, 5120, 8191, 8192, 16384 + 8, 65536]


def token_inputs(seed, M, K, dtype):
    g = np.random.default_rng(seed)
    x = g.standard_normal((M, K), dtype=np.float32) * np.exp(g.standard_normal((M, 1))).astype(np.float32)
    x[:, ::97] *= 20
    if M > 3:
        x[1] = 0
        x[2, K // 2] = np.inf if seed & 1 else np.nan
        x[3] = np.float32(1e-45) * (g.random(K) < 0.5)  # max / 127 underflows
    if M > 5:
        x[4] = np.float32(3e38) * np.sign(x[4] + 1e-9)
        x[5] *= np.float32(1e-39)  # subnormal scale
    return workload.bf16_from_f32(x) if dtype == "bf16" else x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", K_EDGES)
def test_tokens_bitexact(K, dtype):
    for M in (1, 2, 7, 600):
        if M * K > 1 << 22:
            continue
        x = token_inputs(K * 10 + M, M, K, dtype)
        report("quantize_tokens M=%d K=%d %s" % (M, K, dtype))
        codes, scales, sums = dq.quantize_tokens(weights_gpu(x))
        torch().cuda.synchronize()
        o_codes, o_scales, o_sums = tokens_ref(x)
        assert np.array_equal(f32_bits(scales), o_scales.view(np.uint32))
        assert np.array_equal(codes.cpu().numpy(), pad128(o_codes))
        assert np.array_equal(sums.cpu().numpy(), o_sums)


def weights_i8(seed, N, K, bits, asym):
    g = np.random.default_rng(seed)
    w = g.standard_normal((N, K), dtype=np.float32) * np.float32(0.02)
    if asym:
        w = np.abs(w) if seed & 1 else w + np.float32(0.03)
    w = workload.bf16_from_f32(w)
    if asym:
        packed, scales, zeros, u = oracle.quantize_pack_asym(w, bits)
        return packed, scales, zeros, u.astype(np.int64) - zeros[:, None]
    packed, scales, q = oracle.quantize_pack(w, bits)
    return packed, scales, None, np.asarray(q)


def gpu_weights(packed, scales, zeros):
    t = torch()
    return (t.from_numpy(packed.view(np.int32)).cuda(), t.from_numpy(scales).cuda(),
            None if zeros is None else t.from_numpy(np.ascontiguousarray(zeros, np.int32)).cuda())


def assert_product(kind, M, N, K, bits, asym, out, seed, x=None):
    t = torch()
    g = np.random.default_rng(seed + 5)
    if x is None:
        x = workload.bf16_from_f32(g.standard_normal((M, K), dtype=np.float32)
                                   * np.exp(g.standard_normal((M, 1))).astype(np.float32))
    codes, xs, sums = tokens_ref(x)
    packed, scales, zeros, q = weights_i8(seed, N, K, bits, asym)
    P, S, Z = gpu_weights(packed, scales, zeros)
    report("%s_i8 M=%d N=%d K=%d b=%d asym=%s %s" % (kind, M, N, K, bits, asym, out))
    fn = dq.gemv_i8 if kind == "gemv" else dq.gemm_i8
    # one row and one column more than y, filled: what lies behind y stays
    size = M * N
    buf = t.full((size + 256,), 7.0, dtype=t.float32 if out == "f32" else t.bfloat16, device="cuda")
    y = buf[:size].view(M, N)
    fn(t.from_numpy(pad128(codes)).cuda(), t.from_numpy(xs).cuda(), t.from_numpy(sums).cuda(), P, S,
       K, bits, zeros=Z, y=y)
    t.cuda.synchronize()
    assert (buf[size:] == 7.0).all(), "wrote behind y"
    got = y.float().cpu().numpy().astype(np.float64)
    ref = product_ref(codes, xs, q, scales)
    # (float)sum, times sx, times sw: 3 roundings; bf16 rounds once more
    tol = np.abs(ref) * (3 * EPS32 if out == "f32" else EPS_BF16 + 4 * EPS32) * (1 + 1e-6)
    bad = np.abs(got - ref) > tol
    if bad.any():
        m, n = np.argwhere(bad)[0]
        pytest.fail("%d outputs off, first y[%d,%d]=%r ref %r" % (bad.sum(), m, n, got[m, n], ref[m, n]))


@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("bits", range(2, 9))
def test_gemv_i8(bits, asym):
    for M in (1, 2, 3, 4, 5, 8, 9, 16):
        for i, (N, K) in enumerate([(1, 1), (3, 33), (37, 1000), (130, 640), (257, 4096), (20, 5120 + 64)]):
            assert_product("gemv", M, N, K, bits, asym, "bf16" if (M + i) % 3 == 0 else "f32",
                           bits * 1000 + M * 10 + i)


@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("bits", range(2, 9))
def test_gemm_i8(bits, asym):
    for i, (M, N, K) in enumerate([(1, 64, 64), (17, 129, 100), (64, 1, 640), (65, 333, 1027),
                                   (200, 259, 517), (257, 300, 2048), (130, 520, 320)]):
        for out in ("f32", "bf16"):
            assert_product("gemm", M, N, K, bits, asym, out, bits * 1000 + 500 + i)


@pytest.mark.parametrize("bits", [4, 5, 8])
def test_gemm_i8_large_tiles(bits):
    """Enough tiles for every block shape, with ragged last rows and columns."""
    for M, N, K in ((1027, 8200, 384), (300, 16500, 256), (2049, 2100, 640)):
        assert_product("gemm", M, N, K, bits, bits == 5, "f32", bits + M)


@pytest.mark.parametrize("bits", [2, 7, 8])
def test_extreme_sums(bits):
    """Every product of one sign at the largest magnitude and the longest K: the int32 sum
    stays exact (codes +-127 against u at both ends, zero points at both ends)."""
    t = torch()
    K, N = 65536, 6
    top = 2 ** bits - 1
    u = np.zeros((N, K), np.int64)
    u[1], u[3], u[5] = top, top, top // 2
    z = np.array([0, 0, top, top, 1, top], np.int32)
    x = np.full((3, K), 127, np.int8)
    x[1] = -127
    x[2, ::2] = -127
    sums = x.astype(np.int64).sum(1).astype(np.int32)
    packed = pack_codes(u, bits)
    scales = np.ones(N, np.float32)
    ref = x.astype(np.int64) @ (u - z[:, None]).T
    P, S, Z = gpu_weights(packed, scales, z)
    for fn in (dq.gemv_i8, dq.gemm_i8):
        report("extreme sums b=%d %s" % (bits, fn.__name__))
        y = fn(t.from_numpy(x).cuda(), t.ones(3, device="cuda"), t.from_numpy(sums).cuda(), P, S, K, bits, zeros=Z)
        t.cuda.synchronize()
        assert np.array_equal(y.cpu().numpy(), ref.astype(np.float32))


def pack_codes(u, bits):
    N, K = u.shape
    out = np.zeros((N, oracle_row_words(K, bits)), np.uint64)
    for k in range(K):
        pos = k * bits
        w, off = pos >> 5, pos & 31
        v = u[:, k].astype(np.uint64) << np.uint64(off)
        out[:, w] |= v & np.uint64(0xFFFFFFFF)
        if off + bits > 32:
            out[:, w + 1] |= v >> np.uint64(32)
    return out.astype(np.uint32)


def oracle_row_words(K, bits):
    return dq.packed_row_bytes(K, bits) // 4


def test_special_tokens_and_channels():
    """A token with a NaN gives a NaN row, a weight row with one a NaN column; all-zero tokens
    and rows give zeros."""
    t = torch()
    M, N, K = 5, 9, 200
    g = np.random.default_rng(3)
    x = g.standard_normal((M, K)).astype(np.float32)
    x[1, 5] = np.nan
    x[2] = 0
    w = g.standard_normal((N, K)).astype(np.float32)
    w[4, 7] = np.inf
    w[6] = 0
    for bits in (3, 8):
        P, S = dq.quantize_pack(t.from_numpy(w).cuda(), bits)
        tok = dq.quantize_tokens(t.from_numpy(x).cuda())
        for fn in (dq.gemv_i8, dq.gemm_i8):
            y = fn(*tok, P, S, K, bits).cpu().numpy()
            nan = np.zeros((M, N), bool)
            nan[1] = True
            nan[:, 4] = True
            assert np.array_equal(np.isnan(y), nan)
            assert (y[2][[0, 1, 2, 3, 5, 6, 7, 8]] == 0).all() and (y[[0, 2, 3, 4], 6] == 0).all()


def test_one_hot_is_exact():
    """x = one 127 per token, scale 1: the product reads out the codes."""
    t = torch()
    N, K = 70, 384
    for bits in range(2, 9):
        packed, scales, _, q = weights_i8(bits, N, K, bits, False)
        P, S, _ = gpu_weights(packed, np.ones(N, np.float32), None)
        eye = np.zeros((K, K), np.int8)
        np.fill_diagonal(eye, 1)
        one = t.ones(K, device="cuda")
        y = dq.gemm_i8(t.from_numpy(eye).cuda(), one, one.int(), P, S, K, bits)
        assert np.array_equal(y.cpu().numpy(), q.T.astype(np.float32))
        for k in range(0, K, 16):
            y = dq.gemv_i8(t.from_numpy(eye[k:k + 16]).cuda(), one[:16], one[:16].int(), P, S, K, bits)
            assert np.array_equal(y.cpu().numpy(), q.T[k:k + 16].astype(np.float32))


def test_streams_and_graph():
    """On a side stream, and captured in a graph replayed with new inputs between replays."""
    t = torch()
    M, N, K, bits = 6, 200, 700, 6
    packed, scales, _, q = weights_i8(1, N, K, bits, False)
    P, S, _ = gpu_weights(packed, scales, None)
    x = t.randn(M, K, device="cuda").bfloat16()
    want = lambda: dq.gemv_i8(*dq.quantize_tokens(x), P, S, K, bits)
    eager = want()
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        got = want()
    side.synchronize()
    assert t.equal(got, eager)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        y = want()
        ym = dq.gemm_i8(*dq.quantize_tokens(x), P, S, K, bits)
    for i in range(4):
        x.copy_(t.randn(M, K, device="cuda").bfloat16() * (i + 1))
        graph.replay()
        t.cuda.synchronize()
        eager = want()
        assert t.equal(y, eager) and t.equal(ym, eager), i


def test_gemm_and_gemv_agree():
    """Both are exact sums and the same epilogue: identical bits."""
    t = torch()
    for bits in (2, 5, 8):
        for M in (1, 4, 16):
            N, K = 300, 1500
            packed, scales, zeros, _ = weights_i8(bits, N, K, bits, True)
            P, S, Z = gpu_weights(packed, scales, zeros)
            tok = dq.quantize_tokens(t.randn(M, K, device="cuda"))
            assert t.equal(dq.gemv_i8(*tok, P, S, K, bits, zeros=Z), dq.gemm_i8(*tok, P, S, K, bits, zeros=Z))
