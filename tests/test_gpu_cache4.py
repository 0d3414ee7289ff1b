"""The 4-bit key/value cache on the GPU: append bit for bit against the oracle's group
quantizer in the documented storage order, read exactly, attention against fp64 within the
roundings that it makes (serving_ref.attention_tolerance)."""
from __future__ import annotations

import numpy as np
import pytest

import mixed_precision_weight_dq_amd as dq
from gpu_util import bf16_gpu, report, torch, u32
from serving_ref import (Batch, attention_ref, attention_tolerance, bf16, codes_of, group4,
                         key_order, value_order, values, widen, words)

pytestmark = pytest.mark.gpu

GEOMETRY = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


def gpu(a):
    return torch().from_numpy(np.ascontiguousarray(a)).cuda()


def meta(batch):
    return gpu(batch.starts), gpu(batch.lens), gpu(batch.table)


def head_vectors(seed, *shape, special=False):
    """N(0, 1) with hot channels, as fp32; special: zero, subnormal, huge and non-finite groups."""
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape).astype(np.float32)
    x[..., ::41] *= 8
    if special and shape[0] > 6:
        x[1] = 0
        x[2, 0, :32] = np.float32(1e-45)
        x[3] *= np.float32(1e-39)
        x[4] = np.sign(x[4]) * np.float32(3e38)
        x[5, -1, 3] = np.nan
        x[6, 0, -1] = -np.inf
    return x


def place(cache_np, batch, b, codes, scales, order, name):
    """Writes codes [n, H, D] and scales [n, H, G] of sequence b's first n positions."""
    n = codes.shape[0]
    pages, off = batch.places(b, n)
    cache_np[name + "_codes"][pages, :, off] = words(codes, order)
    cache_np[name + "_scales"][pages, :, :, off] = scales


def empty_np(batch, H, D, g, fill=0):
    return {"k_codes": np.full((batch.pages, H, batch.page, D // 8), fill, np.uint32),
            "v_codes": np.full((batch.pages, H, batch.page, D // 8), fill, np.uint32),
            "k_scales": np.full((batch.pages, H, D // g, batch.page), np.nan if fill else 0, np.float32),
            "v_scales": np.full((batch.pages, H, D // g, batch.page), np.nan if fill else 0, np.float32)}


def to_cache(c):
    return dq.Cache4(gpu(c["k_codes"].view(np.int32)), gpu(c["v_codes"].view(np.int32)),
                     gpu(c["k_scales"]), gpu(c["v_scales"]))


def filled(seed, batch, H, D, g):
    """A cache holding random keys and values (unused slots: all-ones codes, NaN scales), and the
    dequantized (k, v) per sequence in fp64."""
    c = empty_np(batch, H, D, g, fill=0xFFFFFFFF)
    kv = []
    for b in range(len(batch.lens)):
        n = max(int(batch.lens[b]), 0)
        pair = []
        for name, order in (("k", key_order(D)), ("v", value_order(D))):
            x = head_vectors(seed * 100 + b * 2 + (name == "v"), n, H, D)
            if n:
                q, s = group4(x, g)
                place(c, batch, b, q, s, order, name)
                pair.append(values(q, s, g).astype(np.float64))
            else:
                pair.append(np.zeros((0, H, D)))
        kv.append(pair)
    return to_cache(c), kv


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,g", GEOMETRY)
def test_append_and_read(D, g, dtype):
    """Decode steps and prompts, strided inputs, special groups; other slots keep their contents."""
    for i, (lens, news, page, H) in enumerate([
            ([1], [1], 16, 1), ([70, 5, 33], [1, 1, 1], 32, 3), ([130, 40, 64, 9], [70, 40, 0, 7], 64, 2),
            ([300], [260], 256, 2), ([17, 16, 15], [9, 16, 2], 16, 5)]):
        batch = Batch(i, lens, news, page)
        T = batch.tokens + 3  # three rows behind the last sequence
        x = head_vectors(i + 10, T, 2 * H + 1, D, special=dtype == "f32" or i == 2)
        bits = bf16(x)
        x = widen(bits) if dtype == "bf16" else x
        fused = bf16_gpu(bits) if dtype == "bf16" else gpu(x)
        k, v = fused[:, 1:1 + H], fused[:, 1 + H:]
        report("cache4_append D=%d g=%d %s lens=%s news=%s page=%d" % (D, g, dtype, lens, news, page))
        c = empty_np(batch, H, D, g, fill=0x12345678)
        for name in ("k_scales", "v_scales"):
            c[name][:] = 5.0
        cache = to_cache(c)
        dq.cache4_append(cache, k, v, *meta(batch))
        torch().cuda.synchronize()
        kq, ks = group4(x[:, 1:1 + H], g)
        vq, vs = group4(x[:, 1 + H:], g)
        want_k, want_v = np.full((T, H, D), 9, np.float32), np.full((T, H, D), 9, np.float32)
        for b in range(len(lens)):
            s, e = batch.starts[b], batch.starts[b + 1]
            pos = np.arange(lens[b] - news[b], lens[b])
            pages, off = batch.table[b, pos // page], pos % page
            for name, q, sc, order in (("k", kq, ks, key_order(D)), ("v", vq, vs, value_order(D))):
                c[name + "_codes"][pages, :, off] = words(q[s:e], order)
                c[name + "_scales"][pages, :, :, off] = sc[s:e]
            want_k[s:e], want_v[s:e] = values(kq[s:e], ks[s:e], g), values(vq[s:e], vs[s:e], g)
        assert np.array_equal(u32(cache.k_codes), c["k_codes"])
        assert np.array_equal(u32(cache.v_codes), c["v_codes"])
        assert np.array_equal(cache.k_scales.cpu().numpy(), c["k_scales"], equal_nan=True)
        assert np.array_equal(cache.v_scales.cpu().numpy(), c["v_scales"], equal_nan=True)
        for kind in (torch().float32, torch().bfloat16):
            ko, vo = (torch().full((T, H, D), 9.0, dtype=kind, device="cuda") for _ in range(2))
            dq.cache4_read(cache, T, *meta(batch), dtype=kind, k=ko, v=vo)
            for got, want in ((ko, want_k), (vo, want_v)):
                want = widen(bf16(want)) if kind == torch().bfloat16 else want
                ok = (got.float().cpu().numpy() == want) | (np.isnan(want) & np.isnan(got.float().cpu().numpy()))
                assert ok.all()


def test_append_skips_what_the_cache_does_not_hold():
    """Positions below 0 or past the table and pages outside the cache: nothing is written for
    them, reads give NaN; the other tokens land."""
    D, g, H, page = 64, 32, 2, 16
    batch = Batch(1, [20, 40, 5], [20, 40, 5], page)
    batch.table[0, 1] = batch.pages  # one past the last page
    batch.table[1, 0] = -1
    lens = batch.lens.copy()
    lens[2] = 3  # two of its five tokens lie below position 0
    lens[1] = 16 * batch.width + 4  # its last four lie past the table
    x = head_vectors(2, batch.tokens, 2 * H, D)
    cache = dq.Cache4.empty(batch.pages, H, D, page, g)
    st, ln, tb = gpu(batch.starts), gpu(lens), gpu(batch.table)
    report("cache4_append with places outside the cache")
    dq.cache4_append(cache, gpu(x)[:, :H], gpu(x)[:, H:], st, ln, tb)
    k, v = dq.cache4_read(cache, batch.tokens, st, ln, tb)
    k, v = k.cpu().numpy(), v.cpu().numpy()
    held = np.ones(batch.tokens, bool)
    held[16:20] = False
    first = int(lens[1]) - 40
    for i in range(40):
        p = first + i
        held[20 + i] = p // page < batch.width and batch.table[1, p // page] >= 0
    held[60:62] = False
    for got, part in ((k, x[:, :H]), (v, x[:, H:])):
        q, s = group4(part, g)
        want = values(q, s, g)
        assert np.array_equal(got[held], want[held])
        assert np.isnan(got[~held]).all()


def run_attention(seed, batch, H, per, D, g, scale=None, q_mul=2.0, max_q=None, max_len=None, tail=2,
                  q=None, prompt=False):
    t = torch()
    cache, kv = filled(seed, batch, H, D, g)
    T = batch.tokens + tail
    if q is None:
        q = np.random.default_rng(seed + 9).standard_normal((T, H * per + 1, D)) * q_mul
    qb = bf16(q)
    out = t.full((T, H * per, D), 9.0, dtype=t.bfloat16, device="cuda")
    dq.cache4_attention(cache, bf16_gpu(qb)[:, 1:], *meta(batch), scale=scale, out=out, max_q=max_q,
                        max_len=max_len)
    t.cuda.synchronize()
    got = out.float().cpu().numpy().astype(np.float64)
    assert (got[batch.tokens:] == 9).all(), "rows behind the last sequence changed"
    scale = D ** -0.5 if scale is None else scale
    q64 = widen(qb)[:batch.tokens, 1:].astype(np.float64)
    ref, W, delta = attention_ref(q64, kv, batch, H * per, scale)
    v_max = max([np.abs(v).max() for _, v in kv if v.size] or [0.0])
    tol = attention_tolerance(ref, W, delta, D, int(batch.lens.max()), v_max, prompt)
    bad = ~(np.abs(got[:batch.tokens] - ref) <= tol)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        pytest.fail("%d of %d off, first %s: %r ref %r tol %r" % (
            bad.sum(), bad.size, at, got[at], ref[at], tol[at]))
    return got[:batch.tokens], ref


@pytest.mark.parametrize("D,g", GEOMETRY)
def test_attention_decode(D, g):
    """One new token per sequence: lengths around tiles and pages, shared heads 1 to 20."""
    for i, (lens, H, per, page) in enumerate([
            ([1], 1, 1, 16), ([1, 2, 15, 16, 17, 31, 32, 33], 2, 4, 16), ([63, 64, 65, 127, 129], 1, 5, 64),
            ([300, 7, 260], 3, 8, 32), ([40, 90], 2, 20, 128), ([513], 2, 16, 256)]):
        batch = Batch(i, lens, [1] * len(lens), page)
        report("cache4_attention decode D=%d g=%d lens=%s H=%d per=%d page=%d" % (D, g, lens, H, per, page))
        run_attention(i + 1, batch, H, per, D, g, max_q=1, max_len=max(lens))


@pytest.mark.parametrize("D,g", [(64, 64), (128, 32), (256, 128)])
def test_attention_several_tokens(D, g):
    """Drafts, prompts from an empty cache and after one, empty sequences, rows that see nothing
    (more new tokens than cached ones), with the launch sized right, too small and by default."""
    for i, (lens, news, H, per, page) in enumerate([
            ([30, 8, 5], [4, 8, 5], 2, 4, 16), ([100, 40, 64, 9], [37, 0, 64, 7], 1, 3, 32),
            ([3, 50], [8, 3], 2, 2, 64), ([0, 20], [2, 1], 1, 8, 16), ([210], [200], 1, 1, 64)]):
        batch = Batch(i, lens, news, page)
        for hints in (dict(max_q=max(news), max_len=max(lens)), dict(max_q=1, max_len=1), {}):
            report("cache4_attention D=%d g=%d lens=%s news=%s H=%d per=%d page=%d %s" % (
                D, g, lens, news, H, per, page, hints))
            got, ref = run_attention(i + 20, batch, H, per, D, g, **hints)
        for b, (n, new) in enumerate(zip(lens, news)):
            if new > n:  # rows that see no position
                s = batch.starts[b]
                assert (got[s:s + new - n] == 0).all()


@pytest.mark.parametrize("D,g", [(64, 32), (128, 32), (128, 128)])
def test_attention_long(D, g):
    """A few thousand positions: many splits and their joining; a batch with short ones beside."""
    batch = Batch(7, [5000, 33, 1500], [1, 1, 2], 64)
    report("cache4_attention long D=%d g=%d" % (D, g))
    run_attention(40, batch, 2, 4, D, g, max_q=2, max_len=5000)
    batch = Batch(8, [9001], [1], 16)
    run_attention(41, batch, 1, 8, D, g, max_q=1, max_len=9001)


@pytest.mark.parametrize("D,g", [(128, 32), (64, 64)])
def test_attention_prompt(D, g):
    """Hundreds of new tokens: tiles of many rows, ragged sequences, a first prompt and a later one."""
    batch = Batch(9, [333, 600, 128], [333, 150, 97], 64)
    report("cache4_attention prompt D=%d g=%d" % (D, g))
    run_attention(50, batch, 2, 3, D, g, max_q=333, max_len=600)


@pytest.mark.parametrize("D,g", GEOMETRY)
def test_attention_prompt_batches(D, g):
    """Enough rows for the kernel of many new tokens (whose rounding of keys and values the bound
    then counts): first prompts and later ones, ragged, empty sequences and rows that see nothing
    among them, tiles of 256 and of 128 rows, the launch sized right and too small."""
    rng = np.random.default_rng(D + g)
    for i, (count, top, H, per, page) in enumerate([(13, 150, 4, 2, 32), (25, 30, 4, 3, 16)]):
        news = [int(n) for n in rng.integers(1, top + 1, count)]
        news[0], news[1], news[2] = top, 0, top // 2
        lens = [n + int(k) for n, k in zip(news, rng.integers(0, 200, count))]
        lens[2] = news[2] - 3  # its first three rows see nothing
        lens[3] = news[3]
        batch = Batch(i, lens, news, page)
        for hints in (dict(max_q=top, max_len=max(lens)), dict(max_q=(top * 2) // 3, max_len=1)):
            report("cache4_attention prompts D=%d g=%d count=%d top=%d %s" % (D, g, count, top, hints))
            got, ref = run_attention(i + 70, batch, H, per, D, g, prompt=True, **hints)
        s = batch.starts[2]
        assert (got[s:s + 3] == 0).all()


def test_attention_prompt_special():
    """The kernel of many new tokens on what it treats apart: NaN groups, pages outside the cache,
    values whose magnitude grows along the sequence, queries far from 1."""
    t = torch()
    D, g, H, per, count, n = 128, 32, 4, 2, 13, 160
    batch = Batch(21, [n] * count, [n] * count, 16)
    k, v = head_vectors(1, count * n, H, D), head_vectors(2, count * n, H, D)
    v *= np.exp2(np.linspace(-30, 20, n)).astype(np.float32)[np.tile(np.arange(n), count), None, None]
    v[3 * n + 70, 1, 40] = np.nan   # sequence 3, head 1, group 1
    k[4 * n + 100, 2, 5] = np.inf   # sequence 4, head 2
    cache = dq.Cache4.empty(batch.pages, H, D, 16, g)
    full = gpu(batch.starts)
    dq.cache4_append(cache, gpu(k), gpu(v), full, gpu(batch.lens), gpu(batch.table))
    kd, vd = dq.cache4_read(cache, count * n, full, gpu(batch.lens), gpu(batch.table))
    kv = [(a, b) for a, b in zip(kd.double().cpu().numpy().reshape(count, n, H, D),
                                 vd.double().cpu().numpy().reshape(count, n, H, D))]
    table = batch.table.copy()
    table[5, 6] = -1  # positions 96 .. 111 of sequence 5
    for mul, scale in ((1.0, None), (2.0 ** 90, 2.0 ** -93)):
        qb = bf16(np.random.default_rng(3).standard_normal((count * n, H * per, D)) * mul)
        report("cache4_attention prompts, special values, q x %g" % mul)
        out = dq.cache4_attention(cache, bf16_gpu(qb), full, gpu(batch.lens), gpu(table), max_q=n,
                                  max_len=n, scale=scale).double().cpu().numpy()
        nan = np.zeros(out.shape, bool)
        nan[3 * n + 70:4 * n, 2:4, 32:64] = True
        nan[4 * n + 100:5 * n, 4:6] = True
        nan[5 * n + 96:6 * n] = True
        assert np.array_equal(np.isnan(out), nan)
        clean = [(np.nan_to_num(a), np.nan_to_num(b)) for a, b in kv]
        ref, W, delta = attention_ref(widen(qb).astype(np.float64), clean, batch, H * per,
                                      D ** -0.5 if scale is None else scale)
        tol = attention_tolerance(ref, W, delta, D, n, np.nanmax(np.abs(vd.cpu().numpy())), True)
        assert (np.abs(out - ref) <= tol)[~nan].all()


def test_attention_logit_range():
    """Peaked and flat softmaxes: scale 0, negative, and logits of several hundred; queries at both
    ends of the bf16 range (all subnormal, near 2^100, mixed)."""
    D, g = 128, 32
    batch = Batch(3, [200, 70], [1, 3], 32)
    for scale in (0.0, -0.3, 1.5):
        report("cache4_attention scale=%g" % scale)
        run_attention(60, batch, 2, 4, D, g, scale=scale, q_mul=3.0)
    for mul, scale in ((1e-39, 1e37), (2.0 ** 100, 2.0 ** -103), (1e-20, 1e19)):
        report("cache4_attention q of magnitude %g" % mul)
        run_attention(61, batch, 2, 4, D, g, scale=scale, q_mul=mul)


@pytest.mark.parametrize("factor", [1e-30, 1e-6, 1e6, 1e30])
def test_attention_value_range(factor):
    """Values of any magnitude, one sequence mixing tokens 2^20 apart: the common power of two
    moves as larger scales come in."""
    t = torch()
    D, g, H = 128, 32, 1
    batch = Batch(4, [150], [1], 16)
    k = head_vectors(1, 150, H, D)
    v = head_vectors(2, 150, H, D) * np.float32(factor)
    v[:75] *= np.float32(2.0 ** -10)
    v[75:100] *= np.float32(2.0 ** 10)
    cache = dq.Cache4.empty(batch.pages, H, D, 16, g)
    st = gpu(np.array([0, 150], np.int32))
    report("cache4_attention values x %g" % factor)
    dq.cache4_append(cache, gpu(k), gpu(v), st, gpu(batch.lens), gpu(batch.table))
    kd, vd = dq.cache4_read(cache, 150, st, gpu(batch.lens), gpu(batch.table))
    kv = [[kd.double().cpu().numpy(), vd.double().cpu().numpy()]]
    qb = bf16(np.random.default_rng(5).standard_normal((1, 4, D)))
    out = dq.cache4_attention(cache, bf16_gpu(qb), *meta(batch)).double().cpu().numpy()
    ref, W, delta = attention_ref(widen(qb).astype(np.float64), kv, batch, 4, D ** -0.5)
    tol = attention_tolerance(ref, W, delta, D, 150, np.abs(kv[0][1]).max())
    assert (np.abs(out - ref) <= tol).all()


def test_attention_bad_metadata():
    """A table that names a page outside the cache, a length past the table: NaN for the queries
    that see it, the other sequences as ever."""
    t = torch()
    D, g, H, per = 64, 32, 2, 4
    batch = Batch(6, [40, 50, 33, 20], [1, 12, 1, 1], 16)
    cache, kv = filled(6, batch, H, D, g)
    q = bf16_gpu(bf16(np.random.default_rng(1).standard_normal((batch.tokens, H * per, D))))
    good = dq.cache4_attention(cache, q, *meta(batch))
    table, lens = batch.table.copy(), batch.lens.copy()
    table[0, 1] = -5
    table[1, 2] = batch.pages  # positions 32 .. 47: the queries at 38 .. 49 all see them
    lens[2] = batch.width * 16 + 1
    report("cache4_attention with bad pages and lengths")
    out = dq.cache4_attention(cache, q, gpu(batch.starts), gpu(lens), gpu(table))
    t.cuda.synchronize()
    s = batch.starts
    assert t.isnan(out[:s[3]]).all()
    assert t.equal(out[s[3]:], good[s[3]:])
    lens[2] = -3  # a negative length holds nothing
    out = dq.cache4_attention(cache, q, gpu(batch.starts), gpu(lens), gpu(batch.table))
    assert (out[s[2]:s[3]] == 0).all() and t.equal(out[:s[2]], good[:s[2]])


def test_attention_nan_groups():
    """A key or value group with a NaN (scale NaN): NaN for the queries that see it and in the
    dimensions that it covers, the ones before it untouched."""
    t = torch()
    D, g, H = 128, 32, 1
    n = 40
    batch = Batch(2, [n], [n], 16)
    k, v = head_vectors(3, n, H, D), head_vectors(4, n, H, D)
    v[25, 0, 70] = np.nan  # group 2: dimensions 64 .. 95
    k[30, 0, 1] = np.inf
    cache = dq.Cache4.empty(batch.pages, H, D, 16, g)
    dq.cache4_append(cache, gpu(k), gpu(v), *meta(batch))
    q = bf16_gpu(bf16(np.random.default_rng(8).standard_normal((n, 2, D))))
    report("cache4_attention with NaN groups")
    out = dq.cache4_attention(cache, q, *meta(batch)).float().cpu().numpy()
    nan = np.zeros((n, 2, D), bool)
    nan[25:, :, 64:96] = True
    nan[30:] = True
    assert np.array_equal(np.isnan(out), nan)


def test_streams_graph_and_workspaces():
    """A decode step (append, attend) captured in a graph, replayed as the sequences grow (starts,
    lens and inputs updated in place), against eager calls; two captures, each with its own
    workspace, replayed in turn; a side stream."""
    t = torch()
    D, g, H, per, B = 128, 32, 2, 4, 3
    batch = Batch(5, [900, 31, 64], [1, 1, 1], 32, width=40)
    table = gpu(np.arange(B * 40, dtype=np.int32).reshape(B, 40))
    c = dq.Cache4.empty(B * 40, H, D, 32, g)
    st = gpu(np.array([0, 1, 2, 3], np.int32))
    lens = gpu(batch.lens)
    full = gpu(np.concatenate([[0], np.cumsum(batch.lens)]).astype(np.int32))
    hist = int(batch.lens.sum())
    dq.cache4_append(c, t.randn(hist, H, D, device="cuda"), t.randn(hist, H, D, device="cuda"), full, lens, table)
    k, v, q = (t.randn(B, n, D, device="cuda").bfloat16() for n in (H, H, H * per))

    def step(cache):
        dq.cache4_append(cache, k, v, st, lens, table)
        return dq.cache4_attention(cache, q, st, lens, table, max_q=1, max_len=1200)

    other = dq.Cache4(*(x.clone() for x in c.tensors))
    eager = dq.Cache4(*(x.clone() for x in c.tensors))
    for cache in (c, other, eager):  # the same contents in all three
        step(cache)
    t.cuda.synchronize()
    graphs = []
    for cache in (c, other):
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            out = step(cache)
        graphs.append((graph, out))
    report("cache4 graphs")
    side = t.cuda.Stream()
    for i in range(4):
        lens += 1
        for x in (k, v, q):
            x.copy_(t.randn_like(x))
        for graph, _ in graphs:
            graph.replay()
        want = step(eager)
        t.cuda.synchronize()
        for _, out in graphs:
            assert t.equal(out, want), i
        side.wait_stream(t.cuda.current_stream())
        with t.cuda.stream(side):
            again = step(eager)
        side.synchronize()
        assert t.equal(again, want)
    need = dq.dq_cache4_attention_workspace(c._c, B, B, H * per, 1, 1200)
    ws = t.full((need + 64,), 3, dtype=t.uint8, device="cuda")
    out = dq.cache4_attention(c, q, st, lens, table, max_q=1, max_len=1200, workspace=ws[:max(need, 16)])
    assert t.equal(out, want) and (ws[max(need, 16):] == 3).all()


def test_repeatable():
    """The same call gives the same bits, alone and beside other sequences."""
    t = torch()
    batch = Batch(11, [2000, 77], [1, 1], 64)
    cache, _ = filled(11, batch, 2, 128, 32)
    q = t.randn(2, 8, 128, device="cuda").bfloat16()
    a = dq.cache4_attention(cache, q, *meta(batch), max_q=1, max_len=2000)
    for _ in range(3):
        assert t.equal(a, dq.cache4_attention(cache, q, *meta(batch), max_q=1, max_len=2000))


def test_long_cache_offsets():
    """Codes past 4 GiB: pages at the far end of a cache whose code arrays hold 2^32 + bytes."""
    t = torch()
    D, g, H, page = 128, 32, 8, 64
    pages = (1 << 32) // (H * page * D // 2) + 40  # 32 KiB of codes per page
    c = dq.Cache4.empty(pages, H, D, page, g)
    n = 150
    table = gpu(np.array([[pages - 1, 3, pages - 7]], np.int32))
    k, v = head_vectors(1, n, H, D), head_vectors(2, n, H, D)
    st, lens = gpu(np.array([0, n], np.int32)), gpu(np.array([n], np.int32))
    report("cache4 beyond 4 GiB")
    dq.cache4_append(c, gpu(k), gpu(v), st, lens, table)
    kd, vd = dq.cache4_read(c, n, st, lens, table)
    kq, ks = group4(k, g)
    assert np.array_equal(kd.cpu().numpy(), values(kq, ks, g))
    q = t.randn(1, H * 2, D, device="cuda").bfloat16()
    one = gpu(np.array([0, 1], np.int32))
    far = dq.cache4_attention(c, q, one, lens, table)
    small = dq.Cache4.empty(3, H, D, page, g)
    for a, b in zip(small.tensors, c.tensors):
        a.copy_(b[table[0].long()])
    near = dq.cache4_attention(small, q, one, lens, gpu(np.array([[0, 1, 2]], np.int32)))
    assert t.equal(far, near)


def test_a_quantized_layer():
    """The operators as a layer's decode step uses them: int8 projections make q, k, v; the cache
    takes k and v; attention; int8 output projection -- against the same steps in fp64 on the
    values that each stage hands over."""
    t = torch()
    hidden, H, per, D, g, bits = 512, 2, 4, 64, 32, 6
    lens, steps = [70, 33, 5], 3
    batch = Batch(13, [n + steps for n in lens], [1, 1, 1], 16)
    table, st = gpu(batch.table), gpu(np.array([0, 1, 2, 3], np.int32))
    rng = np.random.default_rng(2)
    w_qkv = (rng.standard_normal(((H * per + 2 * H) * D, hidden)) * 0.05).astype(np.float32)
    w_out = (rng.standard_normal((hidden, H * per * D)) * 0.05).astype(np.float32)
    pq, sq, zq = dq.quantize_pack_asym(gpu(w_qkv), bits)
    po, so = dq.quantize_pack(gpu(w_out), 8)
    cache = dq.Cache4.empty(batch.pages, H, D, 16, g)
    history = head_vectors(4, sum(lens), 2 * H, D)
    full = gpu(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    dq.cache4_append(cache, gpu(history[:, :H]), gpu(history[:, H:]), full,
                     gpu(np.array(lens, np.int32)), table)
    for step in range(steps):
        now = np.array(lens, np.int32) + step + 1
        x = t.randn(3, hidden, device="cuda").bfloat16()
        tok = dq.quantize_tokens(x)
        qkv = dq.gemv_i8(*tok, pq, sq, hidden, bits, zeros=zq, dtype=t.bfloat16).view(3, -1, D)
        q, k, v = qkv[:, :H * per], qkv[:, H * per:H * per + H], qkv[:, H * per + H:]
        dq.cache4_append(cache, k, v, st, gpu(now), table)
        o = dq.cache4_attention(cache, q, st, gpu(now), table, max_q=1, max_len=int(now.max()))
        y = dq.gemv_i8(*dq.quantize_tokens(o.view(3, -1)), po, so, H * per * D, 8)
        # the projection, exactly
        _, w_hat = dq.unpack_asym(pq, sq, zq, hidden, bits, want_w=True)
        x_hat = tok[0][:, :hidden].double() * tok[1].double()[:, None]
        want = x_hat.cpu() @ w_hat.double().cpu().t()
        got = qkv.reshape(3, -1).double().cpu()
        # w_hat = fl32(q s) rounds each term: 2^-24 of the terms' magnitudes
        mag = x_hat.abs().cpu() @ w_hat.double().abs().cpu().t()
        assert ((got - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -21) + mag * 2.0 ** -23).all()
        # attention over what the cache holds
        all_starts = gpu(np.concatenate([[0], np.cumsum(now)]).astype(np.int32))
        kd, vd = dq.cache4_read(cache, int(now.sum()), all_starts, gpu(now), table)
        cuts = np.cumsum(now)[:-1]
        kv = list(zip(np.split(kd.double().cpu().numpy(), cuts), np.split(vd.double().cpu().numpy(), cuts)))
        at = Batch(13, now, [1, 1, 1], 16)
        ref, W, delta = attention_ref(q.double().cpu().numpy(), kv, at, H * per, D ** -0.5)
        tol = attention_tolerance(ref, W, delta, D, int(now.max()), vd.abs().max().item())
        assert (np.abs(o.double().cpu().numpy() - ref) <= tol).all()
        assert y.shape == (3, hidden) and t.isfinite(y).all()
