"""The int8 activations and the 4-bit cache where their kernels change shape: more sequences than
a wave has lanes, a line of steps that is cut inside the tiles of many new tokens, rows that are
longer than what a thread holds, and quotients at every tie of the quantizer."""
from __future__ import annotations

import numpy as np
import pytest

import mixed_precision_weight_dq_amd as dq
from gpu_util import bf16_gpu, report, torch
from serving_ref import Batch, bf16, group4, tokens_ref, values, widen
from test_gpu_tokens_i8 import assert_product
from test_gpu_cache4 import gpu, head_vectors, meta, run_attention

pytestmark = pytest.mark.gpu


def tie_rows(seed, rows, K, qmax):
    """fp32 rows whose largest magnitude is a and whose other elements lie at the ties of
    v / fl32(a / qmax), up to three steps of fp32 to either side; a from 2^-140 to 2^120."""
    g = np.random.default_rng(seed)
    a = (g.uniform(1, 2, rows) * np.exp2(g.integers(-140, 121, rows))).astype(np.float32)
    s = (a / np.float32(qmax)).astype(np.float32)
    x = ((g.integers(-qmax, qmax, (rows, K)) + 0.5) * s.astype(np.float64)[:, None]).astype(np.float32)
    x = (x.view(np.int32) + g.integers(-3, 4, x.shape, dtype=np.int32)).view(np.float32)
    x = np.clip(x, -a[:, None], a[:, None])
    x[np.arange(rows), g.integers(0, K, rows)] = a
    return x


def test_token_ties():
    """Codes at every tie, fp32 and bf16 (whose few mantissa bits make exact ones common)."""
    x = tie_rows(1, 600, 520, 127)
    report("quantize_tokens at ties")
    for t, ref in ((gpu(x), x), (bf16_gpu(bf16(x)), widen(bf16(x)))):
        codes, scales, sums = dq.quantize_tokens(t)
        want, ws, wsum = tokens_ref(ref)
        assert np.array_equal(scales.cpu().numpy().view(np.uint32), ws.view(np.uint32))
        assert np.array_equal(codes.cpu().numpy()[:, :520], want)
        assert np.array_equal(sums.cpu().numpy(), wsum)


@pytest.mark.parametrize("K", [8191, 8192, 8193, 8200, 16385, 40000])
def test_long_token_rows(K):
    """Rows around and past what a workgroup holds, the largest element in each part of the row."""
    x = np.random.default_rng(K).standard_normal((5, K)).astype(np.float32)
    for m, at in enumerate((0, 8190, K - 1, K // 2, min(8192, K - 1))):
        x[m, at] = 50.0 + m
    report("quantize_tokens K=%d" % K)
    for t, ref in ((gpu(x), x), (bf16_gpu(bf16(x)), widen(bf16(x)))):
        codes, scales, sums = dq.quantize_tokens(t)
        want, ws, wsum = tokens_ref(ref)
        assert np.array_equal(scales.cpu().numpy(), ws)
        assert np.array_equal(codes.cpu().numpy()[:, :K], want)
        assert (codes.cpu().numpy()[:, K:] == 0).all()
        assert np.array_equal(sums.cpu().numpy(), wsum)


@pytest.mark.parametrize("asym", [False, True])
@pytest.mark.parametrize("bits", range(2, 9))
def test_product_shapes(bits, asym):
    """On either side of each choice of the products' kernels: 32 and 33 tokens, one round of
    workgroups of 32 and of 64 tokens, tiles of 64 and of 128 rows, all ragged."""
    for i, (M, N, K) in enumerate([(32, 70, 2200), (33, 70, 2200), (200, 1300, 517), (200, 1500, 517),
                                   (130, 6100, 327), (260, 12000, 200)]):
        assert_product("gemm", M, N, K, bits, asym, "bf16" if i % 2 else "f32", 7000 + 10 * bits + i)


@pytest.mark.parametrize("D,g", [(64, 32), (128, 128), (256, 64)])
def test_cache_ties(D, g):
    H, n = 2, 150
    x = tie_rows(D, n * H * D // g, g, 7).reshape(n, H, D)
    batch = Batch(1, [n], [n], 16)
    for kind in ("f32", "bf16"):
        ref = x if kind == "f32" else widen(bf16(x))
        t = gpu(x) if kind == "f32" else bf16_gpu(bf16(x))
        cache = dq.Cache4.empty(batch.pages, H, D, 16, g)
        report("cache4_append at ties D=%d g=%d %s" % (D, g, kind))
        dq.cache4_append(cache, t, t, *meta(batch))
        k, v = dq.cache4_read(cache, n, *meta(batch))
        want = values(*group4(ref, g), g)
        assert np.array_equal(k.cpu().numpy(), want)
        assert np.array_equal(v.cpu().numpy(), want)


@pytest.mark.parametrize("count", [64, 65, 300])
def test_append_many_sequences(count):
    """Sequences of 0 to 5 new tokens behind what is cached, in one call."""
    D, g, H, page = 128, 32, 2, 16
    rng = np.random.default_rng(count)
    news = [int(n) for n in rng.integers(0, 6, count)]
    lens = [n + int(k) for n, k in zip(news, rng.integers(0, 40, count))]
    batch = Batch(count, lens, news, page)
    x = head_vectors(3, batch.tokens, 2 * H, D)
    cache = dq.Cache4.empty(batch.pages, H, D, page, g)
    for a in cache.tensors:
        a.fill_(-1)
    report("cache4_append count=%d" % count)
    dq.cache4_append(cache, gpu(x)[:, :H], gpu(x)[:, H:], *meta(batch))
    tail = 3
    ko = torch().full((batch.tokens + tail, H, D), 9.0, device="cuda")
    vo = torch().full((batch.tokens + tail, H, D), 9.0, device="cuda")
    dq.cache4_read(cache, batch.tokens + tail, *meta(batch), k=ko, v=vo)
    for got, part in ((ko, x[:, :H]), (vo, x[:, H:])):
        want = values(*group4(part, g), g)
        assert np.array_equal(got[:batch.tokens].cpu().numpy(), want)
        assert (got[batch.tokens:] == 9).all(), "rows behind the last sequence changed"
    # nothing but the new tokens' places was written
    written = np.zeros((batch.pages, page), bool)
    for b, (n, new) in enumerate(zip(lens, news)):
        p = np.arange(n - new, n)
        written[batch.table[b, p // page], p % page] = True
    codes = cache.tensors[0].cpu().numpy()
    assert (codes.transpose(0, 2, 1, 3)[~written] == -1).all()


@pytest.mark.parametrize("D,g", [(64, 64), (128, 32), (256, 128)])
@pytest.mark.parametrize("count", [64, 65, 300])
def test_attention_many_sequences(count, D, g):
    """A decode step of many sequences, some empty, some without a new token."""
    rng = np.random.default_rng(count + D)
    lens = [int(n) for n in rng.integers(0, 150, count)]
    news = [int(n) for n in rng.integers(0, 3, count)]
    batch = Batch(count, lens, news, 16)
    for hints in (dict(max_q=2, max_len=150), dict(max_q=1, max_len=1), dict(max_q=2, max_len=200000)):
        report("cache4_attention count=%d D=%d g=%d %s" % (count, D, g, hints))
        run_attention(5, batch, 1, 4, D, g, **hints)


@pytest.mark.parametrize("D,g", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32),
                                 (256, 64), (256, 128)])
def test_attention_cut_decode(D, g):
    """Few new tokens of short sequences, told of long ones, so that their units are cut: fewer steps
    than workgroups, empty sequences, rows that see nothing, tiles that end inside a head's rows."""
    for i, (lens, news, H, per, page) in enumerate([
            ([1, 2, 15, 16, 17, 31, 32, 33], [1] * 8, 2, 4, 16), ([300, 7, 260], [1] * 3, 3, 8, 32),
            ([513], [1], 2, 16, 256), ([30, 8, 5], [4, 8, 5], 2, 4, 16),
            ([100, 40, 640, 9], [37, 0, 64, 7], 1, 3, 32), ([3, 50], [8, 3], 2, 2, 64),
            ([0, 200], [2, 1], 1, 8, 16)]):
        batch = Batch(i, lens, news, page)
        for hints in (dict(max_q=max(news), max_len=200000), dict(max_q=1, max_len=1)):
            report("cache4_attention cut decode D=%d g=%d lens=%s news=%s %s" % (D, g, lens, news, hints))
            run_attention(i + 400, batch, H, per, D, g, **hints)


# (lens, new tokens, kv heads, query heads of each, page); every call is told of sequences
# long enough for its units to be cut, whatever their lengths are
CUT = [([700], [170], 4, 2, 64),
       ([513, 40, 900], [110, 40, 170], 2, 3, 32),
       ([300, 0, 129, 650], [90, 3, 64, 100], 4, 4, 16)]


@pytest.mark.parametrize("D,g", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32),
                                 (256, 64), (256, 128)])
def test_attention_cut_prompts(D, g):
    """Tiles of many rows cut into stretches: fewer steps than workgroups, empty sequences, rows
    past a sequence's last, more new tokens than cached ones."""
    for i, (lens, news, H, per, page) in enumerate(CUT):
        batch = Batch(i, lens, news, page)
        hints = dict(max_q=max(news), max_len=200000)
        cache = dq.Cache4.empty(1, H, D, page, g)
        need = dq.dq_cache4_attention_workspace(cache._c, len(lens), batch.tokens, H * per,
                                                hints["max_q"], hints["max_len"])
        rows = 128 if D == 256 else 256
        assert need == 256 * 2 * rows * (4 * D + 8)  # the kernel of many rows, cut
        report("cache4_attention cut prompts D=%d g=%d lens=%s news=%s" % (D, g, lens, news))
        run_attention(i + 200, batch, H, per, D, g, prompt=True, **hints)


def test_attention_cut_prompts_many_sequences():
    """More sequences than a wave has lanes, and stretches of several units and parts of units."""
    rng = np.random.default_rng(3)
    count, D, g, H, per = 70, 128, 32, 2, 2
    news = [int(n) for n in rng.integers(0, 71, count)]
    news[0] = 70
    lens = [n + int(k) for n, k in zip(news, rng.integers(0, 300, count))]
    batch = Batch(7, lens, news, 32)
    report("cache4_attention cut prompts of 70 sequences")
    run_attention(300, batch, H, per, D, g, prompt=True, max_q=70, max_len=400)


def test_attention_cut_against_whole():
    """The same prompt over a long cache with its units cut and whole.  Both round their result to
    bf16 (2^-8 each, 2^-7 together), and each weight to 11 bits after it was divided by 2^m, m the
    running maximum: a part that begins elsewhere has another m, so the same weight rounds another
    way, by at most 2^-11 of itself on each side.  Summed: 2 * 2^-11 of W = sum p |v| / sum p, the
    attention over |v| (known to 2^-7 itself); 2^-18 of the largest value for the fp32 sums."""
    t = torch()
    D, g, H, per, n, new = 128, 32, 8, 4, 5000, 400
    batch = Batch(3, [n, n // 2], [new, new], 64)
    total = n + n // 2
    full = gpu(np.array([0, n, total], np.int32))
    cache = dq.Cache4.empty(batch.pages, H, D, 64, g)
    t.manual_seed(1)
    k, v = (t.randn(total, H, D, device="cuda").bfloat16() for _ in range(2))
    dq.cache4_append(cache, k, v, full, gpu(batch.lens), gpu(batch.table))
    q = t.randn(2 * new, H * per, D, device="cuda").bfloat16()
    report("cache4_attention cut against whole")
    cut = dq.cache4_attention(cache, q, *meta(batch), max_q=new, max_len=n).float()
    whole = dq.cache4_attention(cache, q, *meta(batch), max_q=new, max_len=1).float()
    assert not t.equal(cut, whole)  # two ways
    dq.cache4_append(cache, k, v.abs(), full, gpu(batch.lens), gpu(batch.table))
    W = dq.cache4_attention(cache, q, *meta(batch), max_q=new, max_len=1).float()
    tol = 2.0 ** -7 * whole.abs() + 2.0 ** -10 * (1 + 2.0 ** -6) * W + 2.0 ** -18 * v.float().abs().max()
    assert bool(((cut - whole).abs() <= tol).all())
    dq.cache4_append(cache, k, v, full, gpu(batch.lens), gpu(batch.table))
    assert t.equal(cut, dq.cache4_attention(cache, q, *meta(batch), max_q=new, max_len=n).float())


def test_cut_prompt_graphs():
    """Two captures of a cut prompt, each with a workspace of its own, replayed beside eager calls."""
    t = torch()
    D, g, H, per, page = 128, 32, 4, 2, 32
    batch = Batch(2, [600, 330], [170, 60], page)
    cache = dq.Cache4.empty(batch.pages, H, D, page, g)
    total = int(batch.lens.sum())
    full = gpu(np.concatenate([[0], np.cumsum(batch.lens)]).astype(np.int32))
    dq.cache4_append(cache, t.randn(total, H, D, device="cuda"), t.randn(total, H, D, device="cuda"),
                     full, gpu(batch.lens), gpu(batch.table))
    q = t.randn(batch.tokens, H * per, D, device="cuda").bfloat16()
    m = meta(batch)
    call = lambda ws=None: dq.cache4_attention(cache, q, *m, max_q=170, max_len=200000, workspace=ws)
    call()
    t.cuda.synchronize()
    need = dq.dq_cache4_attention_workspace(cache._c, 2, batch.tokens, H * per, 170, 200000)
    assert need > 0
    report("cache4_attention cut prompts in graphs")
    graphs = []
    for _ in range(2):
        ws = t.empty(need, dtype=t.uint8, device="cuda")
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            out = call(ws)
        graphs.append((graph, out, ws))
    for i in range(3):
        q.copy_(t.randn_like(q))
        for graph, _, _ in graphs:
            graph.replay()
        want = call()
        t.cuda.synchronize()
        for _, out, _ in graphs:
            assert t.equal(out, want), i


def test_longest_sequence():
    """2^31 - 2^16 positions, every one of them in the same page, are that page's softmax; one more
    position is refused with NaN.  A lane adds up to 2^18 weights in fp32, each sum within 2^-24:
    2^-6 of W at most, and the roundings of a short sequence beside it."""
    t = torch()
    D, g, page = 64, 64, 256
    n = 2 ** 31 - 2 ** 16
    x = head_vectors(1, page, 2, D)
    cache = dq.Cache4.empty(1, 1, D, page, g)
    one, st = gpu(np.zeros((1, 1), np.int32)), gpu(np.array([0, page], np.int32))
    k, v = gpu(x)[:, :1], gpu(x)[:, 1:]
    dq.cache4_append(cache, k, v, st, gpu(np.array([page], np.int32)), one)
    q = t.randn(1, 2, D, device="cuda").bfloat16()
    row = gpu(np.array([0, 1], np.int32))
    table = t.zeros((1, 2 ** 31 // page), dtype=t.int32, device="cuda")
    report("cache4_attention over 2^31 - 2^16 positions")
    short = dq.cache4_attention(cache, q, row, gpu(np.array([page], np.int32)), one).float()
    long = dq.cache4_attention(cache, q, row, gpu(np.array([n], np.int32)), table, max_q=1, max_len=n).float()
    dq.cache4_append(cache, k, v.abs().contiguous(), st, gpu(np.array([page], np.int32)), one)
    W = dq.cache4_attention(cache, q, row, gpu(np.array([page], np.int32)), one).float()
    assert bool(((long - short).abs() <= 2.0 ** -7 * short.abs() + (2.0 ** -5 + 2.0 ** -9) * W).all())
    over = dq.cache4_attention(cache, q, row, gpu(np.array([n + 1], np.int32)), table, max_q=1, max_len=n)
    assert bool(t.isnan(over).all())


def test_long_cache_offsets_of_prompts():
    """Many new tokens over pages past 4 GiB of codes: the bits of the same call on a cache that
    holds those pages alone, units whole and cut."""
    t = torch()
    D, g, H, per, page, n, new = 128, 32, 8, 2, 64, 700, 200
    pages = (1 << 32) // (H * page * D // 2) + 40  # 32 KiB of codes per page
    c = dq.Cache4.empty(pages, H, D, page, g)
    count = -(-n // page)
    far = np.arange(count, dtype=np.int32)[None] * 3
    far[0, 1::2] = pages - 1 - far[0, 1::2]
    k, v = (t.randn(n, H, D, device="cuda") for _ in range(2))
    st, lens = gpu(np.array([0, n], np.int32)), gpu(np.array([n], np.int32))
    report("cache4 prompts beyond 4 GiB")
    dq.cache4_append(c, k, v, st, lens, gpu(far))
    small = dq.Cache4.empty(count, H, D, page, g)
    for a, b in zip(small.tensors, c.tensors):
        a.copy_(b[gpu(far)[0].long()])
    near = gpu(np.arange(count, dtype=np.int32)[None])
    q = t.randn(new, H * per, D, device="cuda").bfloat16()
    rows = gpu(np.array([0, new], np.int32))
    for max_q, max_len in ((new, 200000), (13 * new, 1)):
        a = dq.cache4_attention(c, q, rows, lens, gpu(far), max_q=max_q, max_len=max_len)
        b = dq.cache4_attention(small, q, rows, lens, near, max_q=max_q, max_len=max_len)
        assert t.equal(a, b) and bool(t.isfinite(a).all())
