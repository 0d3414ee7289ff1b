"""The operators of a drafted step on the GPU, against 64-bit references: rotary positions, keys
rotated into the 4-bit cache, a tree's masks, verification, and kept entries."""
from __future__ import annotations

import numpy as np
import pytest

import mixed_precision_weight_dq_amd as dq
from draft_ref import ancestors, mask_words, random_tree, rotate_ref, rotate_tolerance, verify_ref
from gpu_util import bf16_gpu, report, torch, u32
from serving_ref import Batch, bf16, group4, key_order, value_order, widen, words
from test_gpu_cache4 import GEOMETRY, empty_np, gpu, head_vectors, meta, to_cache

pytestmark = pytest.mark.gpu


def ints(a):
    return gpu(np.asarray(a, np.int32))


def turns_of(rope):
    return rope.turns.cpu().numpy()


# ------------------------------------------------------------------ rotate

ROTATED = [  # tokens, heads, D, dims, interleaved
    (1, 32, 128, 128, False), (1, 1, 64, 64, True), (7, 3, 128, 64, False), (5, 40, 128, 32, True),
    (33, 5, 256, 256, False), (3, 2, 80, 80, True), (4, 3, 96, 24, False), (6, 2, 96, 24, True),
    (2, 1, 2, 2, False), (9, 7, 10, 6, False), (3, 4, 72, 16, True), (130, 9, 128, 128, True), (2, 3, 33, 4, False),
    (2000, 33, 128, 128, False),
]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("case", ROTATED)
def test_rotate(case, kind):
    """Contiguous, in place, as slices (aligned and not), into a strided output, at near and far positions."""
    T, H, D, dims, inter = case
    t = torch()
    scaling = dict(kind="yarn", factor=4, length=512) if dims > 32 else None
    rope = dq.Rope(dims, 10000.0, inter, scaling)
    g = np.random.default_rng(T * D + dims)
    pos = g.integers(0, 5000, T).astype(np.int32)
    pos[:4] = [0, -3, 2 ** 31 - 1, 123456][:T]
    x = (g.standard_normal((T, H, D)) * np.exp(g.standard_normal((T, 1, 1)))).astype(np.float32)
    x = widen(bf16(x)) if kind == "bf16" else x
    xg = bf16_gpu(bf16(x)) if kind == "bf16" else gpu(x)
    ref = rotate_ref(x.astype(np.float64), pos, turns_of(rope), rope.factor, inter)
    tol = rotate_tolerance(x.astype(np.float64), ref, turns_of(rope), rope.factor, inter, kind == "bf16")

    def check(y, what):
        err = np.abs(y.double().cpu().numpy() - ref)
        assert np.all(err <= tol), (what, float((err - tol).max()))

    report("rotate %s %s" % (case, kind))
    check(dq.rotate(rope, xg, ints(pos)), "new")
    y = xg.clone()
    assert dq.rotate(rope, y, ints(pos), out=y) is y
    check(y, "in place")
    for lead, pad in ((2, 8), (1, 3)):  # a slice of more heads, of wider rows
        wide = t.full((T, H + 3, D + pad), 7.0, dtype=xg.dtype, device="cuda")
        part = wide[:, lead:lead + H, :D]
        part.copy_(xg)
        check(dq.rotate(rope, part, ints(pos)), "slice")
        into = t.full((T, H + 1, D + pad), 9.0, dtype=xg.dtype, device="cuda")
        dq.rotate(rope, xg, ints(pos), out=into[:, 1:, :D])
        check(into[:, 1:, :D], "into a slice")
        assert bool((into[:, 0] == 9).all()) and bool((into[:, :, D:] == 9).all())
        dq.rotate(rope, part, ints(pos), out=part)
        check(part, "a slice in place")
        assert bool((wide[:, :lead] == 7).all()) and bool((wide[:, :, D:] == 7).all())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("case", [(700, 33, 72, 16, True), (800, 9, 136, 128, False), (1500, 7, 256, 256, True),
                                  (5000, 9, 80, 64, False), (9000, 33, 64, 64, True), (70000, 1, 24, 16, False),
                                  (700, 33, 72, 18, True)])
def test_rotate_many_tokens(case, kind):
    """Calls that work by pieces of eight dimensions: one head a thread and several, a rest of one piece and of
    many, both orders of pairs; and one whose pairs are no pieces."""
    test_rotate(case, kind)


def test_rotate_special_values():
    """NaN and infinities stay in their pairs; the unrotated rest keeps its bits."""
    t = torch()
    rope = dq.Rope(32)
    x = t.randn(3, 2, 64, device="cuda")
    x[1, 0, 3] = float("nan")
    x[2, 1, 20] = float("inf")
    x[0, 0, 40] = float("nan")
    y = dq.rotate(rope, x, ints([5, 5, 5]))
    bad = ~t.isfinite(y)
    want = t.zeros_like(bad)
    want[1, 0, 3] = want[1, 0, 19] = want[2, 1, 20] = want[2, 1, 4] = want[0, 0, 40] = True
    assert t.equal(bad, want)
    assert t.equal(y[:, :, 32:].view(t.int32), x[:, :, 32:].view(t.int32))


def test_rotate_refuses():
    t = torch()
    rope = dq.Rope(64)
    x, p = t.zeros(3, 2, 64, device="cuda"), ints([0, 1, 2])
    for call in (lambda: dq.rotate(rope, x[..., ::2], p), lambda: dq.rotate(rope, x, p[:2]),
                 lambda: dq.rotate(rope, x, p, out=t.zeros(3, 2, 32, device="cuda")),
                 lambda: dq.rotate(rope, x, p, out=x.bfloat16()), lambda: dq.rotate(rope, x[0], p),
                 lambda: dq.rotate(rope, x, p.cpu())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        dq.rotate(rope, x.half(), p)
    with pytest.raises(TypeError):
        dq.rotate(rope, x, p.long())
    for bad in (x[..., :32], x[:, :, :1].expand(3, 2, 64), x[:1].expand(3, 2, 64)):
        with pytest.raises((dq.DQError, ValueError)):
            dq.rotate(rope, bad, p)
    with pytest.raises(AttributeError):
        rope.dims = 3


# ------------------------------------------------------- append with rotation

def bits_of(cache):
    return [u32(cache.k_codes), u32(cache.v_codes), cache.k_scales.cpu().numpy(), cache.v_scales.cpu().numpy()]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("D,g", GEOMETRY)
def test_append_rotated(D, g, kind):
    """Codes as the oracle's of the key rotated in fp64 and rounded to fp32 (whose last unit may differ in
    1 of 10^7, so a scale by one unit); values, other slots and rows of no sequence as by the plain append."""
    for i, (lens, news, page, H, dims, inter, given) in enumerate([
            ([1], [1], 16, 1, D, False, False), ([70, 5, 33], [1, 1, 1], 32, 3, D, True, False),
            ([130, 40, 64, 9], [70, 40, 0, 7], 64, 2, D // 2, False, True), ([300], [260], 256, 2, D, False, True),
            ([1700], [1600], 64, 9, 16, False, False), ([17, 16, 15], [9, 16, 2], 16, 5, 48, True, False)]):
        batch = Batch(i, lens, news, page)
        T = batch.tokens + 3
        x = head_vectors(i + 10, T, 2 * H + 1, D, special=kind == "f32" or i == 2)
        bits = bf16(x)
        x = widen(bits) if kind == "bf16" else x
        fused = bf16_gpu(bits) if kind == "bf16" else gpu(x)
        k, v = fused[:, 1:1 + H], fused[:, 1 + H:]
        rope = dq.Rope(dims, 10000.0, inter, dict(kind="yarn", factor=4, length=512) if i == 3 else None)
        pos = np.zeros(T, np.int64)
        for b in range(len(lens)):
            pos[batch.starts[b]:batch.starts[b + 1]] = np.arange(lens[b] - news[b], lens[b])
        if given:
            pos = np.random.default_rng(i).integers(-50, 200000, T)
        report("append_rope D=%d g=%d %s lens=%s news=%s dims=%d %s" % (D, g, kind, lens, news, dims, inter))
        c = empty_np(batch, H, D, g, fill=0x12345678)
        for name in ("k_scales", "v_scales"):
            c[name][:] = 5.0
        cache, plain = to_cache(c), to_cache(c)
        dq.cache4_append(plain, k, v, *meta(batch))
        dq.cache4_append(cache, k, v, *meta(batch), rope=rope, positions=ints(pos) if given else None)
        torch().cuda.synchronize()
        with np.errstate(all="ignore"):
            turned = rotate_ref(x[:, 1:1 + H].astype(np.float64), pos, turns_of(rope), rope.factor, inter)
            kq, ks = group4(turned.astype(np.float32), g)
        for b in range(len(lens)):
            s, e = batch.starts[b], batch.starts[b + 1]
            at = np.arange(lens[b] - news[b], lens[b])
            pages, off = batch.table[b, at // page], at % page
            c["k_codes"][pages, :, off] = words(kq[s:e], key_order(D))
            c["k_scales"][pages, :, :, off] = ks[s:e]
        got, same = bits_of(cache), bits_of(plain)
        assert np.array_equal(got[0], c["k_codes"])
        a, b = got[2], c["k_scales"]
        assert np.array_equal(np.isnan(a), np.isnan(b))
        fine = ~np.isnan(b)
        assert np.all(np.abs(a.view(np.int32)[fine].astype(np.int64) - b.view(np.int32)[fine]) <= 1)
        assert np.array_equal(got[1], same[1]) and np.array_equal(got[3], same[3], equal_nan=True)


@pytest.mark.parametrize("inter", [False, True])
def test_append_rotated_by_nothing(inter):
    """At position 0 the plain append's bits; by the formula (0 times an infinity or a NaN) an element that is not
    finite makes its partner NaN, and only that."""
    batch = Batch(3, [40, 9], [40, 5], 16)
    values = widen(bf16(head_vectors(2, batch.tokens, 4, 128, special=True)))
    x = bf16_gpu(bf16(values))
    rope = dq.Rope(128, interleaved=inter)
    turned = values.copy()
    with np.errstate(invalid="ignore"):
        turned[:, :2] = rotate_ref(values[:, :2].astype(np.float64), np.zeros(batch.tokens), turns_of(rope), 1, inter)
    assert np.isnan(turned[:, :2]).sum() == 1  # the partner of the one infinity among the keys
    a, b = (dq.Cache4.empty(batch.pages, 2, 128, 16, 32) for _ in range(2))
    dq.cache4_append(a, gpu(turned[:, :2]), gpu(values[:, 2:]), *meta(batch))
    dq.cache4_append(b, x[:, :2], x[:, 2:], *meta(batch), rope=rope, positions=ints(np.zeros(batch.tokens)))
    for p, q in zip(bits_of(a), bits_of(b)):
        assert np.array_equal(p.view(np.uint32), q.view(np.uint32))


def test_append_rotated_skips_what_the_cache_does_not_hold():
    batch = Batch(3, [40, 20], [12, 8], 16)
    batch.table[0, 2] = batch.pages + 5
    batch.table[1, 0] = -1
    x = bf16_gpu(bf16(head_vectors(2, batch.tokens, 4, 64)))
    a, b = (dq.Cache4.empty(batch.pages, 2, 64, 16, 32) for _ in range(2))
    rope = dq.Rope(64)
    dq.cache4_append(a, dq.rotate(rope, x[:, :2].float(), ints(list(range(28, 40)) + list(range(12, 20)))),
                     x[:, 2:].float(), *meta(batch))
    dq.cache4_append(b, x[:, :2], x[:, 2:], *meta(batch), rope=rope)
    assert np.array_equal(bits_of(a)[2] != 0, bits_of(b)[2] != 0)
    assert np.array_equal(bits_of(a)[1], bits_of(b)[1])


def test_append_rotated_refuses():
    t = torch()
    batch = Batch(3, [4], [4], 16)
    cache = dq.Cache4.empty(batch.pages, 2, 64, 16, 32)
    x = t.zeros(4, 2, 64, device="cuda")
    with pytest.raises(ValueError):
        dq.cache4_append(cache, x, x, *meta(batch), positions=ints([0] * 4))
    with pytest.raises(ValueError):
        dq.cache4_append(cache, x, x, *meta(batch), rope=dq.Rope(64), positions=ints([0] * 3))
    for dims in (24, 80):
        with pytest.raises(dq.DQError):
            dq.cache4_append(cache, x, x, *meta(batch), rope=dq.Rope(dims))


# --------------------------------------------------------------------- tree

def test_draft_tree():
    g = np.random.default_rng(5)
    trees = [[-1], random_tree(g, 40), list(range(-1, 149)), [], random_tree(g, 33, 40), [-1, 0, 5, 2, -7, 4, 99]]
    starts = np.concatenate([[0], np.cumsum([len(x) for x in trees])]).astype(np.int32)
    T = int(starts[-1]) + 2
    parents = np.full(T, 3, np.int32)
    parents[:T - 2] = np.concatenate(trees)
    lens = np.array([1, 100, 150, 7, 40, 7], np.int32)
    for count in (5, 2, 1):
        mask, pos = dq.draft_tree(ints(parents), ints(starts), ints(lens), words=count)
        only, none = dq.draft_tree(ints(parents), ints(starts), words=count)
        assert none is None and torch().equal(only, mask)
        mask, pos = mask.cpu().numpy(), pos.cpu().numpy()
        for b, tree in enumerate(trees):
            s, e = starts[b], starts[b + 1]
            sees = ancestors(tree)
            assert np.array_equal(mask[s:e], mask_words(sees, count)), (b, count)
            if len(tree):
                assert np.array_equal(pos[s:e], lens[b] - len(tree) + sees.sum(1) - 1)
        assert not mask[T - 2:].any() and not pos[T - 2:].any()
    mask, _ = dq.draft_tree(ints(parents), ints(starts))
    assert mask.shape == (T, -(-T // 32))


def test_rows_past_the_largest_tree():
    """A sequence's rows from 4096 on are roots that no path reaches: chains of 4095, 4096 and 4200 rows."""
    sizes = [4095, 4200, 4096, 3]
    starts = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    T = int(starts[-1])
    parents = np.concatenate([np.arange(-1, n - 1) for n in sizes]).astype(np.int32)
    lens = (np.array(sizes) + 50).astype(np.int32)
    mask, pos = dq.draft_tree(ints(parents), ints(starts), ints(lens), words=132)
    mask, pos = mask.cpu().numpy(), pos.cpu().numpy()
    for b, n in enumerate(sizes):
        i = np.arange(n)
        sees = (i[None] <= i[:, None]) & (i[:, None] < 4096) | (i[None] == i[:, None])
        assert np.array_equal(mask[starts[b]:starts[b + 1]], mask_words(sees, 132))
        assert np.array_equal(pos[starts[b]:starts[b + 1]], 50 + np.where(i < 4096, i, 0))
    g = np.random.default_rng(2)
    probs = softmax(g.standard_normal((T, 9)))
    ids, u = g.integers(0, 9, T).astype(np.int32), np.zeros(T, np.float32)
    u[starts[:-1]] = 0.5
    path, accepted, drawn = (x.cpu().numpy() for x in dq.verify_drafts(gpu(probs), ints(ids), ints(parents),
                                                                       ints(starts), gpu(u)))
    assert list(accepted) == [min(n, 4096) for n in sizes]
    for b, n in enumerate(sizes):
        i = np.arange(n)
        assert np.array_equal(path[starts[b]:starts[b + 1]], np.where(i < 4096, i, -1))
        last = probs[starts[b] + accepted[b] - 1].astype(np.float64)  # its child, if any, is past the tree
        assert drawn[b] == np.flatnonzero(np.cumsum(last) > 0.5 * last.sum())[0]
    # children of one row, all refused: each id once, as far as the tree reaches
    parents[starts[1]:starts[2]] = 0
    ids[starts[1]:starts[2]] = np.where(np.arange(4200) < 4096, np.arange(4200) % 3, 5)
    u[starts[1]:starts[2]] = 0.999999
    probs[starts[1]] = np.float32(1 / 9)
    _, accepted, drawn = dq.verify_drafts(gpu(probs), ints(ids), ints(parents), ints(starts), gpu(u))
    assert int(accepted[1]) == 1 and int(drawn[1]) == 8
    u[starts[1]] = 0.4  # of ids 3 .. 8
    _, accepted, drawn = dq.verify_drafts(gpu(probs), ints(ids), ints(parents), ints(starts), gpu(u))
    assert int(accepted[1]) == 1 and int(drawn[1]) == 5


# ------------------------------------------------------------------- verify

def softmax(x):
    p = np.exp(x - x.max(-1, keepdims=True))
    return (p / p.sum(-1, keepdims=True)).astype(np.float32)


def drafts(seed, sizes, V, chain):
    """Probabilities, draft probabilities, ids, parents, starts, uniforms of a batch."""
    g = np.random.default_rng(seed)
    T = sum(sizes)
    logits = g.standard_normal((T, V)) * 2
    probs, q = softmax(logits), softmax(logits + g.standard_normal((T, V)) * 0.5)
    starts = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    parents = np.concatenate([list(range(-1, n - 1)) if chain else random_tree(g, n) for n in sizes if n]).astype(np.int32)
    ids = np.zeros(T, np.int32)
    for b, n in enumerate(sizes):
        for i in range(n):
            row = starts[b] + max(int(parents[starts[b] + i]), 0)
            w = q[row].astype(np.float64)
            ids[starts[b] + i] = g.choice(V, p=w / w.sum())
    return probs, q, ids, parents, starts, g.random(T).astype(np.float32)


def check_verify(probs, q, ids, parents, starts, u, draft, pad=0):
    t = torch()
    T, V = probs.shape
    want = verify_ref(probs, ids, parents, starts, u, q if draft else None)

    def rows(a):  # rows with a gap between them
        w = t.full((T, V + pad), 0.5, device="cuda")
        w[:, :V] = gpu(a)
        return w[:, :V]

    got = dq.verify_drafts(rows(probs), ints(ids), ints(parents), ints(starts), gpu(np.asarray(u, np.float32)),
                           draft_probs=rows(q) if draft else None)
    for a, b, name in zip(got, want, ("path", "accepted", "next")):
        a = a.cpu().numpy()
        end = int(starts[-1]) if name == "path" else len(a)
        assert np.array_equal(a[:end], b[:end]), (name, a, b)
    return want


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("V", [1, 2, 63, 64, 65, 2047, 2048, 2049, 5000, 33001])
def test_verify(V, draft):
    for seed, sizes in enumerate([[1], [2, 5, 0, 1, 9], [64, 65, 130, 3], [0, 0, 4]]):
        if V > 6000 and sum(sizes) > 100:
            sizes = [17, 5]
        report("verify V=%d draft=%d %s" % (V, draft, sizes))
        for chain in (True, False):
            check_verify(*drafts(seed + V, sizes, V, chain), draft, pad=seed)


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("V", [255, 256, 257, 1023, 1024, 1025, 1281])
def test_verify_ends_of_stretches(V, draft):
    """The last ids of a stretch, of a wave's and of a thread's part of it: drawn with random numbers near 1."""
    for seed in range(3):
        probs, q, ids, parents, starts, u = drafts(100 * seed + V, [1, 3, 4, 1, 2], V, True)
        u[starts[:-1]] = [1 - 2.0 ** -24, 0.9999, 0.75, 0.25, 0.0]
        check_verify(probs, q, ids, parents, starts, u, draft)


@pytest.mark.parametrize("draft", [False, True])
def test_verify_everything_taken_or_refused(draft):
    probs, q, ids, parents, starts, u = drafts(7, [40, 70, 6], 300, True)
    assert list(check_verify(probs, probs if draft else q, ids, parents, starts, u * 0, draft)[1]) == [40, 70, 6]
    near = np.full_like(u, 1 - 2.0 ** -24)
    check_verify(probs, q, ids, parents, starts, near, draft)
    check_verify(probs, q, ids, parents, starts, np.ones_like(u), draft)
    assert list(check_verify(probs, q, ids, parents, starts, u * np.nan, draft)[1]) == [1, 1, 1]


@pytest.mark.parametrize("draft", [False, True])
def test_verify_odd_inputs(draft):
    """Ids outside the vocabulary, siblings with one id, parents that are no row, equal distributions (nothing
    left: the target's own are drawn from), rows without any probability."""
    probs, q, ids, parents, starts, u = drafts(3, [30, 100, 12, 5], 70, False)
    ids[4::7] = [-1, 70, 2 ** 31 - 1, -5][:1] * len(ids[4::7])
    ids[5::9] = 70
    parents[20] = 25
    parents[21] = -9
    parents[22] = 10 ** 9
    ids[31:100] = ids[31:100] % 3
    check_verify(probs, q, ids, parents, starts, u, draft)
    parents[31:130] = 0   # one row's children, more than a wave has lanes, many of them with one id
    check_verify(probs, q, ids, parents, starts, np.maximum(u, 0.9), draft)
    check_verify(probs, probs, ids, parents, starts, u, draft)
    ids[1] = 75  # refused though p and q are the same
    check_verify(probs, probs, ids, parents, starts, u, draft)
    probs[30] = 0
    probs[:, ::3] = 0
    check_verify(probs, q, ids, parents, starts, u, draft)
    one = np.zeros_like(probs)
    one[np.arange(len(one)), ids.clip(0, 69)] = 1
    check_verify(one, q, ids, parents, starts, u, draft)


@pytest.mark.parametrize("draft", [False, True])
def test_verify_many_stretches(draft):
    """A vocabulary of more stretches than a wave has lanes, the drawn token in the first, the last and between."""
    V = 2048 * 66 + 5
    probs, q, ids, parents, starts, u = drafts(3, [3, 2, 2, 1], V, not draft)
    u[starts[:-1]] = [0.0, 0.999999, 0.97, 0.5]
    last = check_verify(probs, q, ids, parents, starts, u, draft)[2]
    assert last[1] > 2048 * 60


def test_verify_rows_far_apart():
    """Rows 2^29 elements apart: offsets past 32 bits."""
    t = torch()
    probs, q, ids, parents, starts, u = drafts(3, [5, 4], 777, True)
    far = t.empty((8 << 29) + 777, device="cuda")
    rows = far.as_strided((9, 777), (1 << 29, 1))
    rows.copy_(gpu(probs))
    for draft in (None, gpu(q)):
        got = dq.verify_drafts(rows, ints(ids), ints(parents), ints(starts), gpu(u), draft_probs=draft)
        want = verify_ref(probs, ids, parents, starts, u, None if draft is None else q)
        for a, b in zip(got, want):
            assert np.array_equal(a.cpu().numpy(), b)


def test_verify_not_finite_ends():
    """Probabilities that are not finite give some token or none, and touch nothing else."""
    probs, q, ids, parents, starts, u = drafts(3, [6, 3], 5000, True)
    for bad in (np.nan, np.inf, -1.0):
        p = probs.copy()
        p[:, ::2] = bad
        for draft in (None, gpu(q)):
            path, accepted, drawn = dq.verify_drafts(gpu(p), ints(ids), ints(parents), ints(starts), gpu(u),
                                                     draft_probs=draft)
            assert bool(((drawn >= -1) & (drawn < 5000)).all())
            assert bool(((accepted >= 1) & (accepted <= 6)).all())


# --------------------------------------------------------------------- keep

@pytest.mark.parametrize("D,g", GEOMETRY)
def test_keep(D, g):
    """Accepted entries in front of the call's positions, everything else untouched."""
    r = np.random.default_rng(D + g)
    for lens, news, page, H in (([9], [9], 16, 1), ([100, 40, 70, 33], [64, 7, 0, 20], 16, 3), ([300], [200], 64, 9)):
        batch = Batch(D, lens, news, page)
        c = {n: r.integers(0, 2 ** 32, a.shape, np.uint32) if a.dtype == np.uint32 else r.random(a.shape, np.float32)
             for n, a in empty_np(batch, H, D, g).items()}
        cache = to_cache(c)
        path, accepted = np.full(batch.tokens + 1, -1, np.int32), []
        for b, n in enumerate(news):
            a = int(r.integers(1, n + 1)) if n else 0
            rows = np.sort(r.choice(n, a, replace=False)) if n else []
            path[batch.starts[b]:batch.starts[b] + a] = rows
            accepted.append(a + (3 if b == 1 else 0))  # beyond the rows: entries of -1
        want = {n: a.copy() for n, a in c.items()}
        for b, n in enumerate(news):
            for j in range(min(accepted[b], n)):
                row = path[batch.starts[b] + j]
                if row < j:
                    continue
                src, dst = lens[b] - n + row, lens[b] - n + j
                ps, pd = batch.table[b, src // page], batch.table[b, dst // page]
                for name in want:
                    if "codes" in name:
                        want[name][pd, :, dst % page] = c[name][ps, :, src % page]
                    else:
                        want[name][pd, :, :, dst % page] = c[name][ps, :, :, src % page]
        report("keep D=%d g=%d %s" % (D, g, lens))
        dq.cache4_keep(cache, *meta(batch), ints(path), ints(accepted))
        for x, name in zip(bits_of(cache), ("k_codes", "v_codes", "k_scales", "v_scales")):
            assert np.array_equal(x, want[name]), name


def test_keep_leaves_bad_entries():
    """Paths that point back, out of the rows or nowhere, counts below 0, pages outside the cache."""
    batch = Batch(1, [30, 30, 20], [10, 10, 10], 16)
    batch.table[2, 0] = batch.pages
    cache = dq.Cache4.empty(batch.pages, 2, 64, 16, 32)
    cache.k_codes.random_()
    cache.k_scales.uniform_()
    before = bits_of(cache)
    path = np.array([0, 0, 1, -1, 10, 99, 2 ** 31 - 1, 7, -2 ** 31, 9] + [5] * 10 + list(range(10)), np.int32)
    path[27] = 8
    dq.cache4_keep(cache, *meta(batch), ints(path), ints([10, -4, 10]))
    after = bits_of(cache)
    # path[7] = 7 stays; sequence 2's row 8 replaces row 7, position 17, which the cache holds
    page, moved = batch.table[2, 1], before[0].copy()
    moved[page, :, 1] = before[0][page, :, 2]
    assert np.array_equal(after[0], moved)


def test_keep_refuses():
    batch = Batch(1, [30], [10], 16)
    cache = dq.Cache4.empty(batch.pages, 2, 64, 16, 32)
    with pytest.raises(ValueError):
        dq.cache4_keep(cache, *meta(batch), ints([0] * 10), ints([1, 2]))
    with pytest.raises(TypeError):
        dq.cache4_keep(cache, *meta(batch), ints([0] * 10).long(), ints([1]))
