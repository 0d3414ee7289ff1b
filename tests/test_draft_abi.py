"""Refusals of the drafted step's entry points (returned on the host before any HIP call, so these
run without a GPU; the fake device addresses are never dereferenced), and the frequencies of
``Rope`` against their definitions."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

import mixed_precision_weight_dq_amd as dq
from test_serving_abi import A, BATCH, MIS, structs


def rope(**kw):
    return dq.DQRope(**{**dict(turns=A, dims=32, interleaved=0, factor=1.0), **kw})


def rotate(**kw):
    r = rope(**{n: kw.pop(n) for n in ("turns", "dims", "interleaved", "factor") if n in kw})
    return dq.dq_rotate(kw.pop("rope", r), **{**dict(
        x=A, dtype=dq.DQ_BF16, tokens=3, heads=2, head_dim=64, x_token_stride=128, x_head_stride=64,
        positions=A, out=A, out_token_stride=128, out_head_stride=64), **kw})


def append(**kw):
    c, b = structs(kw)
    r = rope(**{n: kw.pop(n) for n in ("turns", "dims", "interleaved", "factor") if n in kw})
    return dq.dq_cache4_append_rope(c, b, **{**dict(k=A, v=A, dtype=dq.DQ_BF16, tokens=3, k_stride=128,
                                                    v_stride=128, rope=r, positions=A), **kw})


def keep(**kw):
    c, b = structs(kw)
    return dq.dq_cache4_keep(c, b, **{**dict(path=A, accepted=A, tokens=3), **kw})


def attend(**kw):
    c, b = structs(kw)
    return dq.dq_cache4_tree_attention(c, b, **{**dict(
        q=A, tokens=3, q_stride=256, q_heads=4, mask=A, mask_words=1, scale=0.1, max_q=1, max_len=30,
        out=A, workspace=A, workspace_bytes=1 << 40), **kw})


def tree(**kw):
    return dq.dq_draft_tree(**{**dict(parents=A, starts=A, lens=A, count=2, tokens=3, words=1, mask=A,
                                      positions=A), **kw})


def verify(**kw):
    return dq.dq_verify_drafts(**{**dict(
        probs=A, probs_stride=100, draft_probs=A, draft_stride=100, ids=A, parents=A, starts=A, uniforms=A,
        tokens=3, count=2, vocab=100, path=A, accepted=A, next=A, workspace=A, workspace_bytes=1 << 40), **kw})


def test_rotate_refusals():
    for name in ("x", "positions", "out", "turns", "rope"):
        assert rotate(**{name: None if name == "rope" else 0}) == dq.DQ_ERR_NULL
    for kw in (dict(dims=0), dict(dims=3), dict(dims=66), dict(dims=4098), dict(head_dim=16), dict(head_dim=4097),
               dict(tokens=0), dict(tokens=1 << 31), dict(heads=0), dict(heads=1025), dict(x_token_stride=127),
               dict(x_head_stride=63), dict(out_token_stride=100), dict(out_head_stride=-64),
               dict(x_token_stride=(1 << 32) + 8), dict(x_head_stride=0)):
        assert rotate(**kw) == dq.DQ_ERR_SHAPE, kw
    assert rotate(dtype=2) == rotate(dtype=-1) == dq.DQ_ERR_DTYPE
    for factor in (math.nan, math.inf):
        assert rotate(factor=factor) == dq.DQ_ERR_VALUE
    for kw in (dict(x=A + 1), dict(out=A + 1), dict(x=A + 2, dtype=dq.DQ_F32), dict(positions=A + 2),
               dict(turns=MIS)):
        assert rotate(**kw) == dq.DQ_ERR_ALIGN, kw


@pytest.mark.parametrize("call", [append, keep, attend])
def test_cache_refusals(call):
    for name in ("k_codes", "v_codes", "k_scales", "v_scales", "starts", "lens", "table"):
        assert call(**{name: 0}) == dq.DQ_ERR_NULL
        assert call(**{name: A + (2 if name in BATCH else 4)}) == dq.DQ_ERR_ALIGN
    for kw in (dict(head_dim=32), dict(page_size=8), dict(page_size=48), dict(group=16), dict(group=128),
               dict(kv_heads=0), dict(kv_heads=1025), dict(pages=0), dict(count=0), dict(count=65536),
               dict(table_width=0), dict(table_width=(1 << 24) + 1), dict(tokens=0), dict(tokens=1 << 31)):
        assert call(**kw) == dq.DQ_ERR_SHAPE, kw


def test_append_refusals():
    for name in ("k", "v", "turns"):
        assert append(**{name: 0}) == dq.DQ_ERR_NULL
    assert append(k=MIS) == append(v=MIS) == append(positions=A + 2) == append(turns=MIS) == dq.DQ_ERR_ALIGN
    assert append(dtype=2) == dq.DQ_ERR_DTYPE
    for kw in (dict(k_stride=127), dict(v_stride=120), dict(dims=0), dict(dims=24), dict(dims=80), dict(dims=2)):
        assert append(**kw) == dq.DQ_ERR_SHAPE, kw
    assert append(factor=math.inf) == dq.DQ_ERR_VALUE


def test_keep_refusals():
    assert keep(path=0) == keep(accepted=0) == dq.DQ_ERR_NULL
    assert keep(path=A + 2) == keep(accepted=A + 1) == dq.DQ_ERR_ALIGN


def test_attention_refusals():
    assert attend(q=0) == attend(out=0) == attend(mask=0) == dq.DQ_ERR_NULL
    assert attend(q=MIS) == attend(out=MIS) == attend(workspace=MIS) == attend(mask=A + 2) == dq.DQ_ERR_ALIGN
    for kw in (dict(q_heads=0), dict(q_heads=3), dict(q_heads=1026), dict(q_stride=255), dict(max_q=0),
               dict(max_len=0), dict(mask_words=0), dict(mask_words=65537)):
        assert attend(**kw) == dq.DQ_ERR_SHAPE, kw
    for scale in (math.inf, math.nan, 3e38):
        assert attend(scale=scale) == dq.DQ_ERR_VALUE


def test_attention_workspace():
    c, _ = structs({})
    size = lambda **kw: dq.dq_cache4_tree_attention_workspace(
        c, **{**dict(count=2, tokens=2, q_heads=4, max_q=1, max_len=100), **kw})
    for kw in (dict(count=0), dict(tokens=0), dict(q_heads=3), dict(max_q=0), dict(max_len=0)):
        assert size(**kw) == 0
    long = size(max_len=1 << 17)
    assert long >= size() >= 0
    if long:
        kw = dict(count=2, tokens=2, max_len=1 << 17)
        assert attend(workspace=0, **kw) == dq.DQ_ERR_NULL
        assert attend(workspace_bytes=long - 1, **kw) == dq.DQ_ERR_SHAPE


@pytest.mark.parametrize("heads,q_heads", [(1, 1), (1, 1024), (8, 64), (1024, 1024)])
@pytest.mark.parametrize("max_q", [1, 1000, 2 ** 31 - 1, 2 ** 62])
@pytest.mark.parametrize("max_len", [1, 10 ** 6, 2 ** 62])
def test_attention_workspace_bounds(heads, q_heads, max_q, max_len):
    """No product of sizes wraps: at most two tiles of 128 rows of 256 for each of 2048 workgroups."""
    p = ctypes.c_void_p(4096)
    c = dq.DQCache4(p, p, p, p, 2 ** 31 - 1, heads, 256, 16, 32)
    for count in (1, 65535):
        need = dq.dq_cache4_tree_attention_workspace(c, count, 2 ** 31 - 1, q_heads, max_q, max_len)
        assert 0 <= need <= 2 * 2048 * 128 * (4 * 256 + 8)


def test_tree_refusals():
    for name in ("parents", "starts", "mask", "lens"):
        assert tree(**{name: 0}) == dq.DQ_ERR_NULL
    for name in ("parents", "starts", "mask", "lens", "positions"):
        assert tree(**{name: A + 2}) == dq.DQ_ERR_ALIGN
    for kw in (dict(count=0), dict(count=65536), dict(tokens=0), dict(tokens=1 << 31), dict(words=0),
               dict(words=65537)):
        assert tree(**kw) == dq.DQ_ERR_SHAPE


def test_verify_refusals():
    for name in ("probs", "ids", "parents", "starts", "uniforms", "path", "accepted", "next", "workspace"):
        assert verify(**{name: 0}) == dq.DQ_ERR_NULL
    for name in ("probs", "draft_probs", "ids", "parents", "starts", "uniforms", "path", "accepted", "next"):
        assert verify(**{name: A + 2}) == dq.DQ_ERR_ALIGN
    assert verify(workspace=A + 8) == dq.DQ_ERR_ALIGN
    for kw in (dict(count=0), dict(count=65536), dict(tokens=0), dict(vocab=0), dict(vocab=(1 << 24) + 1),
               dict(probs_stride=99), dict(draft_stride=99), dict(probs_stride=(1 << 32) + 1),
               dict(workspace_bytes=0)):
        assert verify(**kw) == dq.DQ_ERR_SHAPE, kw
    assert dq.dq_verify_drafts_workspace(0, 10) == dq.dq_verify_drafts_workspace(1, 0) == 0
    assert dq.dq_verify_drafts_workspace(3, 128000) >= 3 * 8


def turns_of(dims, base, scaling):
    turns, factor = dq._rope_turns(dims, base, scaling)
    return np.array(turns) * 2 * np.pi, factor


def test_rope_frequencies():
    """Each kind at pairs whose value its definition gives directly."""
    plain, f = turns_of(128, 10000.0, None)
    assert f == 1 and len(plain) == 64
    np.testing.assert_allclose(plain, 10000.0 ** (-np.arange(64) / 64), rtol=1e-14)
    np.testing.assert_allclose(turns_of(128, 10000.0, dict(kind="linear", factor=4))[0], plain / 4, rtol=1e-14)
    ntk, _ = turns_of(128, 10000.0, dict(kind="ntk", factor=4))
    assert ntk[0] == plain[0]                                  # the fastest pair as it was,
    np.testing.assert_allclose(ntk[-1], plain[-1] / 4, rtol=1e-12)  # the slowest as if divided
    yarn, f = turns_of(128, 10000.0, dict(kind="yarn", factor=8, length=4096))
    assert f == pytest.approx(0.1 * math.log(8) + 1, rel=1e-15)
    rounds = 4096 * plain / (2 * np.pi)
    assert np.array_equal(yarn[rounds > 40], plain[rounds > 40])
    np.testing.assert_allclose(yarn[rounds < 0.8], plain[rounds < 0.8] / 8, rtol=1e-14)
    between = yarn / plain
    assert np.all(np.diff(between) <= 1e-15) and np.any((between > 0.2) & (between < 0.9))
    bands, f = turns_of(128, 500000.0, dict(kind="bands", factor=8, length=8192, low=1, high=4))
    slow = turns_of(128, 500000.0, None)[0]
    rounds = 8192 * slow / (2 * np.pi)
    assert f == 1 and np.array_equal(bands[rounds >= 4], slow[rounds >= 4])
    np.testing.assert_allclose(bands[rounds <= 1], slow[rounds <= 1] / 8, rtol=1e-14)
    w = (rounds - 1) / 3
    mid = (w > 0) & (w < 1)
    assert mid.any()
    np.testing.assert_allclose(bands[mid], (1 - w[mid]) * slow[mid] / 8 + w[mid] * slow[mid], rtol=1e-13)
    some, f = turns_of(4, 100.0, dict(kind="list", divisors=[1, 5], amplitude=1.25))
    assert f == 1.25
    np.testing.assert_allclose(some, [1.0, 0.1 / 5], rtol=1e-14)


@pytest.mark.parametrize("dims,base,scaling", [
    (7, 1e4, None), (0, 1e4, None), (4098, 1e4, None), (64, 1.0, None), (64, math.inf, None),
    (64, 1e4, dict(kind="other")), (64, 1e4, dict(factor=2)), (64, 1e4, dict(kind="linear")),
    (64, 1e4, dict(kind="linear", factor=0)), (64, 1e4, dict(kind="linear", factor=2, fast=3)),
    (2, 1e4, dict(kind="ntk", factor=2)), (64, 1e4, dict(kind="yarn", factor=2)),
    (64, 1e4, dict(kind="yarn", factor=2, length=100, fast=1, slow=2)),
    (64, 1e4, dict(kind="bands", factor=2, length=100, low=4, high=4)),
    (64, 1e4, dict(kind="list", divisors=[1.0])), (4, 1e4, dict(kind="list", divisors=[1.0, -1.0]))])
def test_rope_refusals(dims, base, scaling):
    with pytest.raises((ValueError, dq.DQError)):
        dq._rope_turns(dims, base, scaling)


def test_torch_layer_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        dq.Rope(64, device="cpu")
    i = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: dq.rotate(None, torch.zeros(3, 2, 64), i),
                 lambda: dq.draft_tree(i, i),
                 lambda: dq.verify_drafts(torch.zeros(3, 10), i, i, i, torch.zeros(3))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        dq.rotate(None, [1.0], i)


def test_rule_keeps_the_targets_law():
    """Over a grid of random numbers, the token behind the root is distributed as the target's: for
    candidates tried in order, and for one drawn from the draft's probabilities."""
    from draft_ref import verify_ref
    p = np.array([0.1, 0.2, 0.3, 0.4])
    q = np.array([0.4, 0.3, 0.2, 0.1])
    probs = np.stack([p] * 3).astype(np.float32)
    n = 40
    grid = (np.arange(n) + 0.5) / n
    got = np.zeros(4)
    for a in grid:          # two candidates, the first the less likely, then the drawn one
        for c in grid:
            for z in grid:
                path, k, last = verify_ref(probs, [9, 1, 3], [-1, 0, 0], [0, 3], [z, a, c])
                got[[1, 3][path[1] - 1] if k[0] == 2 else last[0]] += 1
    np.testing.assert_allclose(got / n ** 3, p, atol=1.5 / n)
    got = np.zeros(4)
    draft = np.stack([q] * 2).astype(np.float32)
    for token in range(4):  # a chain of one, its token drawn from q
        for a in grid:
            for z in grid:
                path, k, last = verify_ref(probs[:2], [9, token], [-1, 0], [0, 2], [z, a], draft)
                got[token if k[0] == 2 else last[0]] += q[token] / n ** 2
    np.testing.assert_allclose(got, p, atol=1.5 / n)
