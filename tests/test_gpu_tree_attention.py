"""Attention of drafted trees over the 4-bit cache against fp64 within the roundings that it makes
(draft_ref.tree_tolerance), and a whole drafted step."""
from __future__ import annotations

import numpy as np
import pytest

import mixed_precision_weight_dq_amd as dq
from draft_ref import ancestors, mask_words, random_tree, tree_ref, tree_tolerance
from gpu_util import bf16_gpu, report, torch
from serving_ref import Batch, bf16, widen
from test_gpu_cache4 import GEOMETRY, filled, gpu, head_vectors, meta

pytestmark = pytest.mark.gpu


def masks(g, batch, kind):
    """sees[b] bool [new, new]: trees, or any bits at all (some rows without one)."""
    out = []
    for n in batch.news:
        if kind == "tree":
            out.append(ancestors(random_tree(g, n)) if n else np.zeros((0, 0), bool))
        else:
            m = g.random((n, n)) < g.choice([0.1, 0.5, 0.9], (n, 1))
            m[::3] &= g.random((len(m[::3]), 1)) < 0.5
            out.append(m)
    return out


def bits(g, batch, sees, words, tokens):
    """Mask words; bits past a sequence's rows, and rows of no sequence, are noise."""
    m = g.integers(-2 ** 31, 2 ** 31, (tokens, words)).astype(np.int32)
    for b, s in enumerate(sees):
        n = len(s)
        keep = np.ones((1, words * 32), bool)
        keep[:, :n] = False
        noise = mask_words(keep.repeat(n, 0), words)
        rows = slice(batch.starts[b], batch.starts[b + 1])
        m[rows] = (m[rows] & noise) | mask_words(s, words)
    return m


def attend(cache, kv, batch, H, per, sees, seed=0, scale=None, words=None, q_mul=1.0, extra=0, **kw):
    """The call's output, the reference and its tolerance."""
    g = np.random.default_rng(seed)
    D = cache.head_dim
    T = batch.tokens + extra
    qb = bf16(g.standard_normal((T, H * per, D)) * q_mul)
    words = words or -(-max(batch.news) // 32)
    m = bits(g, batch, sees, words, T)
    out = dq.cache4_tree_attention(cache, bf16_gpu(qb), *meta(batch), gpu(m), scale=scale, **kw)
    torch().cuda.synchronize()
    q = widen(qb).astype(np.float64)
    args = tree_ref(q, kv, batch, H * per, D ** -0.5 if scale is None else scale, sees)
    return out.double().cpu().numpy(), args[0], tree_tolerance(*args, D, int(batch.lens.max()))


def check(got, ref, tol, rows=None):
    bad = ~(np.abs(got - ref) <= tol)
    if rows is not None:
        bad = bad[rows]
    assert not bad.any(), "%d of %d off, first %s" % (bad.sum(), bad.size, np.argwhere(bad)[0])


CASES = [  # lens, news, page, kv heads, query heads of one
    ([1], [1], 16, 1, 1), ([2, 40], [2, 9], 16, 2, 4), ([33, 64, 5, 70], [33, 31, 0, 32], 32, 1, 2),
    ([200], [100], 64, 2, 1), ([130, 700, 31], [65, 7, 31], 16, 2, 5), ([1500], [3], 256, 1, 8),
]


@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("D,g", GEOMETRY)
def test_tree_attention(D, g, kind):
    for i, (lens, news, page, H, per) in enumerate(CASES):
        batch = Batch(i, lens, news, page)
        report("tree attention D=%d g=%d %s lens=%s news=%s" % (D, g, kind, lens, news))
        cache, kv = filled(i + 3, batch, H, D, g)
        sees = masks(np.random.default_rng(i), batch, kind)
        got, ref, tol = attend(cache, kv, batch, H, per, sees, seed=i, words=1 + -(-max(news) // 32),
                               scale=-0.07 if i == 1 else (0.0 if i == 3 else None), q_mul=3.0)
        check(got, ref, tol)


@pytest.mark.parametrize("hints", [dict(max_q=1, max_len=1), dict(max_q=64, max_len=100000), dict()])
def test_tree_attention_sizes_of_the_launch(hints):
    """Hints size the launch only: right with ones too small, too large, or none."""
    batch = Batch(1, [900, 64, 3000, 10], [40, 64, 5, 10], 64)
    cache, kv = filled(9, batch, 2, 128, 32)
    sees = masks(np.random.default_rng(2), batch, "tree")
    check(*attend(cache, kv, batch, 2, 4, sees, **hints))


def test_tree_attention_many_sequences():
    """More sequences than a wave has lanes, ragged, some empty."""
    g = np.random.default_rng(0)
    lens = [int(n) for n in g.integers(1, 120, 90)]
    news = [int(min(n, g.integers(0, 20))) for n in lens]
    lens[7], news[7] = 0, 0
    batch = Batch(4, lens, news, 16)
    cache, kv = filled(5, batch, 2, 64, 32)
    check(*attend(cache, kv, batch, 2, 2, masks(g, batch, "any"), extra=0))


def test_rows_of_no_sequence_stay():
    batch = Batch(4, [30, 20], [4, 3], 16)
    cache, kv = filled(5, batch, 1, 64, 32)
    sees = masks(np.random.default_rng(1), batch, "tree")
    out = torch().full((batch.tokens + 4, 2, 64), 7.0, dtype=torch().bfloat16, device="cuda")
    got, ref, tol = attend(cache, kv, batch, 1, 2, sees, extra=4, out=out)
    check(got, ref, tol, slice(0, batch.tokens))
    assert (got[batch.tokens:] == 7).all()


def test_chain_is_causal():
    """A chain's mask gives what cache4_attention gives, within both roundings."""
    batch = Batch(4, [500, 90], [20, 33], 64)
    cache, kv = filled(5, batch, 2, 128, 64)
    sees = [np.tril(np.ones((n, n), bool)) for n in batch.news]
    got, ref, tol = attend(cache, kv, batch, 2, 4, sees, seed=3)
    check(got, ref, tol)
    qb = bf16(np.random.default_rng(3).standard_normal((batch.tokens, 8, 128)))
    other = dq.cache4_attention(cache, bf16_gpu(qb), *meta(batch)).double().cpu().numpy()
    check(got, other, 2 * tol)


def test_words_that_end_early():
    """Rows without a bit are seen by none, themselves not by themselves."""
    batch = Batch(4, [150, 80], [100, 64], 16)
    cache, kv = filled(5, batch, 1, 64, 64)
    sees = masks(np.random.default_rng(1), batch, "any")
    cut = [s & (np.arange(len(s)) < 64) for s in sees]
    check(*attend(cache, kv, batch, 1, 3, cut, words=2))


@pytest.mark.parametrize("D,g", [(64, 32), (128, 128), (256, 64)])
def test_hidden_positions_have_no_part(D, g):
    """NaN scales, codes of other magnitudes and pages outside the cache, at drafted positions that
    rows do not see: those rows keep their bits; rows that see a NaN are NaN (a key's everywhere, a value's in its
    group's dimensions)."""
    t = torch()
    lens, n = [70, 40], 24
    batch = Batch(4, lens, [n, n], 16)
    cache, kv = filled(5, batch, 2, D, g)
    rng = np.random.default_rng(2)
    sees = [ancestors(random_tree(rng, n)) for _ in lens]
    qb = bf16_gpu(bf16(rng.standard_normal((batch.tokens, 4, D))))
    mask = gpu(np.concatenate([mask_words(s, 1) for s in sees]))
    call = lambda c: dq.cache4_tree_attention(c, qb, *meta(batch), mask).double().cpu().numpy()
    first = call(cache)
    row = 9
    for what in ("key", "value", "large", "small", "page"):
        changed = dq.Cache4(*(x.clone() for x in cache.tensors))
        table = batch.table.copy()
        for b in range(2):
            at = lens[b] - n + row
            page, off = int(batch.table[b, at // 16]), at % 16
            if what == "key":
                changed.k_scales[page, :, 0, off] = float("nan")
            elif what == "value":
                changed.v_scales[page, :, 0, off] = float("nan")
            elif what == "page":
                pass
            else:
                f = 1e18 if what == "large" else 1e-18
                changed.k_scales[page, :, :, off] *= f
                changed.v_scales[page, :, :, off] *= f
        hidden = [~s[:, row] for s in sees]
        if what == "page":  # a whole page of drafted positions: the rows that see none of it
            for b in range(2):
                last = (lens[b] - 1) // 16
                table[b, last] = -1
                gone = np.arange(n) + lens[b] - n >= 16 * last
                hidden[b] = ~(sees[b] & gone).any(1)
        keep_table, batch.table = batch.table, table
        got = call(changed)
        batch.table = keep_table
        hidden = np.concatenate(hidden)
        assert hidden.any() and (~hidden).any()
        assert np.array_equal(got[hidden], first[hidden]), what
        if what in ("key", "page"):
            assert np.isnan(got[~hidden]).all()
        if what == "value":
            assert np.isnan(got[~hidden][..., :g]).all() and np.array_equal(got[~hidden][..., g:], first[~hidden][..., g:])


def test_bad_lengths():
    """A length past the table, or past what the attention takes, makes its sequence NaN; fewer cached tokens than
    rows leave the first without a position."""
    t = torch()
    batch = Batch(4, [60, 40, 6, 50], [8, 8, 8, 8], 16)
    cache, kv = filled(5, batch, 1, 64, 32)
    sees = [np.tril(np.ones((8, 8), bool))] * 4
    mask = gpu(np.concatenate([mask_words(s, 1) for s in sees]))
    qb = bf16_gpu(bf16(np.random.default_rng(1).standard_normal((32, 2, 64))))
    call = lambda: dq.cache4_tree_attention(cache, qb, *meta(batch), mask).double().cpu().numpy()
    first = call()
    assert np.isfinite(first).all() and not first[16:18].any() and first[18:24].any()
    width = batch.table.shape[1]
    for bad in (width * 16 + 1, 2 ** 31 - 1, 2 ** 31 - 2 ** 16 + 1):
        batch.lens[0] = bad
        got = call()
        assert np.isnan(got[:8]).all() and np.array_equal(got[8:], first[8:]), bad
    batch.lens[0] = -5
    got = call()
    assert not got[:8].any() and np.array_equal(got[8:], first[8:])


def test_values_far_apart():
    """Magnitudes that grow and fall along the sequence, zero tokens and zero groups among them."""
    from serving_ranges import with_zeros
    for D, g in ((64, 32), (128, 64), (256, 128)):
        for f in (1e-5, 1e-13, 1e6):
            batch = Batch(7, [220, 150], [40, 12], 16)
            H = 1
            cache = dq.Cache4.empty(batch.pages, H, D, 16, g)
            full = gpu(np.array([0, 220, 370], np.int32))
            x = head_vectors(3, 370, 2 * H, D)
            x[60:120] *= f
            x[200:260] *= f
            for a, b in ((0, 220), (220, 370)):
                x[a:b] = with_zeros(x[a:b], b - a, g)
            dq.cache4_append(cache, gpu(x[:, :H]), gpu(x[:, H:]), full, gpu(batch.lens), gpu(batch.table))
            k, v = dq.cache4_read(cache, 370, full, gpu(batch.lens), gpu(batch.table))
            kv = [(k[a:b].double().cpu().numpy(), v[a:b].double().cpu().numpy()) for a, b in ((0, 220), (220, 370))]
            sees = masks(np.random.default_rng(2), batch, "any")
            check(*attend(cache, kv, batch, H, 4, sees, q_mul=1.0 if f < 1 else 1e-6))


def test_refusals():
    t = torch()
    batch = Batch(4, [30], [4], 16)
    cache, _ = filled(5, batch, 1, 64, 32)
    q = t.zeros(4, 2, 64, dtype=t.bfloat16, device="cuda")
    m = t.zeros(4, 1, dtype=t.int32, device="cuda")
    for call in (lambda: dq.cache4_tree_attention(cache, q, *meta(batch), m[:3]),
                 lambda: dq.cache4_tree_attention(cache, q, *meta(batch), m[:, 0]),
                 lambda: dq.cache4_tree_attention(cache, q, *meta(batch), m, out=q[:3]),
                 lambda: dq.cache4_tree_attention(cache, q, *meta(batch), m.cpu())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        dq.cache4_tree_attention(cache, q, *meta(batch), m.long())
    with pytest.raises(TypeError):
        dq.cache4_tree_attention(cache, q.float(), *meta(batch), m)
    with pytest.raises(dq.DQError):
        dq.cache4_tree_attention(cache, q, *meta(batch), m[:, :0])


def step_inputs(seed=0):
    """Three sequences with cached contexts and trees of drafts."""
    g = np.random.default_rng(seed)
    contexts, news = [90, 33, 200], [20, 7, 33]
    batch = Batch(seed, [c + n + 5 for c, n in zip(contexts, news)], news, 16)
    batch.lens = np.array([c + n for c, n in zip(contexts, news)], np.int32)
    parents = [random_tree(g, n) for n in news]
    return g, contexts, batch, parents


def test_a_whole_step():
    """Rotated queries and keys, the tree's attention, verification and kept entries, together; then the next
    token's attention over the kept cache is that over one filled with the accepted tokens alone."""
    t = torch()
    t.manual_seed(5)
    g, contexts, batch, parents = step_inputs()
    H, per, D, V = 2, 4, 128, 500
    rope = dq.Rope(D)
    starts, lens, table = meta(batch)
    cache = dq.Cache4.empty(batch.pages, H, D, 16, 32)
    old = t.randn(sum(contexts), 2 * H, D, device="cuda").bfloat16()
    first = gpu(np.concatenate([[0], np.cumsum(contexts)]).astype(np.int32))
    held = gpu(np.array(contexts, np.int32))
    dq.cache4_append(cache, old[:, :H], old[:, H:], first, held, table, rope=rope)

    flat = gpu(np.concatenate(parents).astype(np.int32))
    mask, positions = dq.draft_tree(flat, starts, lens, words=2)
    qkv = t.randn(batch.tokens, (per + 2) * H, D, device="cuda").bfloat16()
    k, v = qkv[:, per * H:(per + 1) * H], qkv[:, (per + 1) * H:]
    q = dq.rotate(rope, qkv[:, :per * H], positions)
    dq.cache4_append(cache, k, v, starts, lens, table, rope=rope, positions=positions)
    out = dq.cache4_tree_attention(cache, q, starts, lens, table, mask, max_q=33, max_len=240)
    kd, vd = dq.cache4_read(cache, int(batch.lens.sum()),
                            gpu(np.concatenate([[0], np.cumsum(batch.lens)]).astype(np.int32)), lens, table)
    cuts = np.cumsum(batch.lens)[:-1]
    kv = list(zip(np.split(kd.double().cpu().numpy(), cuts), np.split(vd.double().cpu().numpy(), cuts)))
    args = tree_ref(q.double().cpu().numpy(), kv, batch, H * per, D ** -0.5, [ancestors(p) for p in parents])
    check(out.double().cpu().numpy(), args[0], tree_tolerance(*args, D, int(batch.lens.max())))

    probs = t.softmax(t.randn(batch.tokens, V, device="cuda") * 4, -1)
    best = t.topk(probs, 40, dim=-1).indices
    ids, seen = np.zeros(batch.tokens, np.int32), {}
    for b, p in enumerate(parents):
        for i in range(1, len(p)):
            row = int(batch.starts[b]) + p[i]
            ids[batch.starts[b] + i] = best[row, seen.get(row, 0)]
            seen[row] = seen.get(row, 0) + 1
    u = t.rand(batch.tokens, device="cuda") * 0.7
    path, accepted, drawn = dq.verify_drafts(probs, gpu(ids), flat, starts, u)
    dq.cache4_keep(cache, starts, lens, table, path, accepted)

    acc = accepted.cpu().numpy()
    assert acc.max() > 2 and (drawn.cpu().numpy() >= 0).all()
    rows = np.concatenate([int(batch.starts[b]) + path.cpu().numpy()[batch.starts[b]:batch.starts[b] + a]
                           for b, a in enumerate(acc)])
    rows = t.from_numpy(rows).cuda()
    other = dq.Cache4.empty(batch.pages, H, D, 16, 32)
    dq.cache4_append(other, old[:, :H], old[:, H:], first, held, table, rope=rope)
    kept = gpu(np.concatenate([[0], np.cumsum(acc)]).astype(np.int32))
    now = held + accepted
    dq.cache4_append(other, k[rows].contiguous(), v[rows].contiguous(), kept, now, table, rope=rope)
    one, nq = gpu(np.arange(4, dtype=np.int32)), t.randn(3, H * per, D, device="cuda").bfloat16()
    for c in (cache, other):
        dq.cache4_append(c, k[:3], v[:3], one, now + 1, table, rope=rope)
    a, b = (dq.cache4_attention(c, nq, one, now + 1, table, max_q=1, max_len=240) for c in (cache, other))
    assert t.equal(a, b)


def test_streams_and_graphs():
    """On another stream, and captured: replays with eager work between them, two graphs each with a
    workspace of its own replayed side by side."""
    t = torch()
    batch = Batch(4, [3000, 500], [30, 12], 64)
    cache, kv = filled(5, batch, 2, 128, 32)
    g = np.random.default_rng(1)
    sees = masks(g, batch, "tree")
    starts, lens, table = meta(batch)
    mask = gpu(np.concatenate([mask_words(s, 1) for s in sees]))
    q = bf16_gpu(bf16(g.standard_normal((batch.tokens, 8, 128))))
    probs = t.softmax(t.randn(batch.tokens, 3001, device="cuda") * 3, -1)
    parents = gpu(np.concatenate([random_tree(g, n) for n in batch.news]).astype(np.int32))
    ids = t.argmax(probs, -1).to(t.int32)
    u = t.rand(batch.tokens, device="cuda")
    rope = dq.Rope(128)
    pos = t.arange(batch.tokens, device="cuda", dtype=t.int32)

    def run():
        r = dq.rotate(rope, q, pos)
        return (r, dq.cache4_tree_attention(cache, r, starts, lens, table, mask, max_q=30, max_len=3000),
                *dq.verify_drafts(probs, ids, parents, starts, u), *dq.draft_tree(parents, starts, lens))

    want = run()
    t.cuda.synchronize()
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        other = run()
    side.synchronize()
    for a, b in zip(other, want):
        assert t.equal(a, b)
    graphs = []
    for _ in range(2):
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            outs = run()
        graphs.append((graph, outs))
    for _ in range(4):
        for graph, outs in graphs:
            for x in outs:
                x.zero_()
        t.cuda.synchronize()
        for i, (graph, outs) in enumerate(graphs):
            with t.cuda.stream(side if i else t.cuda.current_stream()):
                graph.replay()
        t.cuda.synchronize()
        for graph, outs in graphs:
            for a, b in zip(outs, want):
                assert t.equal(a, b)
        eager = run()
        t.cuda.synchronize()
        for a, b in zip(eager, want):
            assert t.equal(a, b)


@pytest.mark.parametrize("D,g", GEOMETRY)
@pytest.mark.parametrize("hints", [dict(max_q=64, max_len=200000), dict(max_q=8, max_len=300), dict(max_q=20, max_len=4000)])
def test_every_shape_of_the_launch(D, g, hints):
    """Whole units and stretches (what the hints ask for), on lengths that are none of those:
    several tiles, several masked steps of a wave, units that end inside a stretch."""
    batch = Batch(3, [700, 333, 150], [290, 21, 150], 32)
    cache, kv = filled(11, batch, 2, D, g)
    sees = masks(np.random.default_rng(6), batch, "any")
    report("tree attention D=%d g=%d %s" % (D, g, hints))
    check(*attend(cache, kv, batch, 2, 3, sees, seed=5, **hints))


def test_repeated_calls_give_the_same_bits():
    batch = Batch(3, [5000, 900], [30, 12], 64)
    cache, _ = filled(11, batch, 4, 128, 32)
    sees = masks(np.random.default_rng(6), batch, "tree")
    mask = gpu(np.concatenate([mask_words(s, 1) for s in sees]))
    q = torch().randn(batch.tokens, 16, 128, device="cuda").bfloat16()
    call = lambda: dq.cache4_tree_attention(cache, q, *meta(batch), mask, max_q=30, max_len=5000)
    first = call()
    for _ in range(5):
        assert torch().equal(call(), first)


@pytest.mark.parametrize("D,g", [(64, 64), (128, 32), (256, 128)])
@pytest.mark.parametrize("f", [1e-5, 1e-9, 1e-25])
def test_a_row_keeps_its_bits_beside_larger_drafts(D, g, f):
    """Drafts (and their zero groups) far larger than what other rows see: the bound is relative to what a row
    sees.  Context far smaller than the drafts, none at all, and drafts apart from each other."""
    from serving_ranges import with_zeros
    for lens, news in (([90, 40], [60, 40]), ([300, 33], [20, 2])):
        batch = Batch(7, lens, news, 16)
        H, n = 2, sum(lens)
        cache = dq.Cache4.empty(batch.pages, H, D, 16, g)
        full = gpu(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
        x = head_vectors(3, n, 2 * H, D)
        at = 0
        for length, new in zip(lens, news):
            x[at:at + length] *= f
            x[at + length - new:at + length:3] /= f
            x[at:at + length] = with_zeros(x[at:at + length], length, g)
            at += length
        dq.cache4_append(cache, gpu(x[:, :H]), gpu(x[:, H:]), full, gpu(batch.lens), gpu(batch.table))
        k, v = dq.cache4_read(cache, n, full, gpu(batch.lens), gpu(batch.table))
        cuts = np.cumsum(lens)[:-1]
        kv = list(zip(np.split(k.double().cpu().numpy(), cuts), np.split(v.double().cpu().numpy(), cuts)))
        sees = []
        for new in news:  # rows see their own kind of drafts: the larger or the smaller ones
            i = np.arange(new)
            sees.append((i[:, None] % 3 == 0) == (i[None] % 3 == 0))
            sees[-1] &= i[None] <= i[:, None]
        report("tree attention, larger drafts D=%d f=%g %s" % (D, f, lens))
        check(*attend(cache, kv, batch, H, 3, sees))


def test_pages_past_4_gib():
    """Codes, scales and kept entries at offsets past 32 bits."""
    t = torch()
    pages, H, D, P, g = 150000, 8, 128, 64, 32
    codes = lambda: t.empty(pages, H, P, D // 8, dtype=t.int32, device="cuda")
    scales = lambda: t.empty(pages, H, D // g, P, device="cuda")
    big = dq.Cache4(codes(), codes(), scales(), scales())
    batch = Batch(3, [300, 70], [30, 9], P)
    small = dq.Cache4.empty(batch.pages, H, D, P, g)
    move = pages - 1 - batch.table  # the same pages from the far end
    rope = dq.Rope(D)
    T = int(batch.lens.sum())
    full = gpu(np.concatenate([[0], np.cumsum(batch.lens)]).astype(np.int32))
    x = t.randn(T, 2 * H, D, device="cuda").bfloat16()
    starts, lens, table = meta(batch)
    far = gpu(move.astype(np.int32))
    q = t.randn(batch.tokens, 4 * H, D, device="cuda").bfloat16()
    sees = masks(np.random.default_rng(6), batch, "tree")
    mask = gpu(np.concatenate([mask_words(s, 1) for s in sees]))
    path = gpu(np.array([0, 3, 5, 7] + [-1] * 26 + [0, 8] + [-1] * 7, np.int32))
    outs = []
    for cache, tab in ((small, table), (big, far)):
        dq.cache4_append(cache, x[:, :H], x[:, H:], full, lens, tab, rope=rope)
        out = dq.cache4_tree_attention(cache, q, starts, lens, tab, mask)
        dq.cache4_keep(cache, starts, lens, tab, path, gpu(np.array([4, 2], np.int32)))
        outs.append((out, *dq.cache4_read(cache, T, full, lens, tab)))
    for a, b in zip(*outs):
        assert t.equal(a, b)


@pytest.mark.parametrize("D,g", GEOMETRY)
@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("H,per,max_len", [(8, 8, 30000), (8, 2, 4000), (2, 3, 30000)])
def test_several_units_of_a_workgroup(D, g, kind, H, per, max_len):
    """Stretches that hold several units, whole ones and parts: short sequences under hints of long ones."""
    batch = Batch(60, [35, 160, 115, 17, 17, 565, 130], [2, 32, 100, 17, 1, 65, 2], 32)
    cache, kv = filled(160, batch, H, D, g)
    sees = masks(np.random.default_rng(60), batch, kind)
    report("tree attention, several units D=%d g=%d %s H=%d per=%d" % (D, g, kind, H, per))
    check(*attend(cache, kv, batch, H, per, sees, seed=60, words=5, max_q=100, max_len=max_len))
