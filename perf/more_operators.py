"""Cases that measure the operators of a drafted decode step over the 4-bit cache.

A serving step that drafts several tokens ahead runs, around the projections:

* ``rotate``    -- rotary positions of the queries: half and interleaved pairs, part of a
                   head, frequencies scaled for long contexts;
* ``append``    -- keys rotated at their positions and quantized, with the values, into the
                   paged 4-bit cache in one call (and read back, which is how the stored
                   values are seen);
* ``attention`` -- attention of a tree of drafted tokens: each sees the cached context and
                   its own ancestors;
* ``verify``    -- the drafts against the target's probabilities, from given random numbers:
                   the accepted path and the token drawn behind it;
* ``keep``      -- the accepted path's entries of the cache moved next to the context (and
                   read back).

``run`` computes each in elementary torch operations, or, where ``own`` is true, through the
package.  Shapes: heads of 64, 128 or 256, eight or fewer kv heads, vocabularies of 1000 to
128000, trees of 2 to 64 drafted tokens.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token's queries of a decode step
        dict(name="rotate-1x32x128", op="rotate", t=1, h=32, d=128, r=128, inter=False, base=10000.0,
             kind="none", s=1.0, far=6000, dtype="bf16"),
        # a prompt's queries, half of each head, a context stretched to sixteen times its length
        dict(name="rotate-6000x40x128-yarn", op="rotate", t=6000, h=40, d=128, r=64, inter=True,
             base=500000.0, kind="yarn", s=16.0, far=100000, dtype="bf16"),
        # a decode step's new keys and values of 32 sequences
        dict(name="append-32x1", op="append", b=32, q=1, len=2000, hq=32, hkv=8, d=128, g=32,
             page=64, r=128, inter=False, base=10000.0, kind="none", s=1.0, out="f32"),
        # prompts into the cache, frequencies scaled by bands
        dict(name="append-3x2500-bands", op="append", b=3, q=2500, len=2900, hq=64, hkv=8, d=128,
             g=64, page=64, r=128, inter=False, base=500000.0, kind="bands", s=8.0, out="bf16"),
        # small drafts of a few sequences, narrow heads, small pages
        dict(name="attention-8x6-1100", op="attention", b=8, q=6, len=1100, hq=16, hkv=4, d=64,
             g=64, page=16),
        # one long sequence and a large tree
        dict(name="attention-1x64-65000", op="attention", b=1, q=64, len=65000, hq=32, hkv=8, d=128,
             g=32, page=64),
        # a ragged batch with trees of up to 24
        dict(name="attention-24x24-6000", op="attention", b=24, q=24, len=6000, hq=40, hkv=8, d=128,
             g=32, page=64),
        # one sequence's chain, with the draft's own probabilities
        dict(name="verify-1x6x32000", op="verify", b=1, q=6, v=32000, tree=False),
        # trees of candidates, an odd vocabulary
        dict(name="verify-16x32x50001-tree", op="verify", b=16, q=32, v=50001, tree=True),
        # a batch of chains over a large vocabulary
        dict(name="verify-48x7x128000", op="verify", b=48, q=7, v=128000, tree=False),
        # the accepted tokens of one sequence's draft
        dict(name="keep-1x16", op="keep", b=1, q=16, len=3000, hq=32, hkv=8, d=128, g=32, page=64),
        # those of a batch
        dict(name="keep-64x64", op="keep", b=64, q=64, len=2000, hq=32, hkv=8, d=128, g=32, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rope(rng, d):
    return dict(r=rng.choice([d, d, d // 2, d // 4]), inter=rng.random() < 0.5,
                base=rng.choice([10000.0, 500000.0, 1000000.0]),
                kind=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                s=rng.choice([2.0, 4.0, 8.0, 16.0]))


def draw(rng):
    op = rng.choice(["rotate", "append", "attention", "attention", "verify", "keep"])
    if op == "rotate":
        d = rng.choice([64, 80, 96, 128, 128, 256])
        return dict(op=op, t=_log(rng, 1, 1700), h=_log(rng, 1, 36), d=d, **_draw_rope(rng, d),
                    far=_log(rng, 10, 1000000), dtype=rng.choice(["bf16", "f32"]))
    if op == "verify":
        tree = rng.random() < 0.5
        return dict(op=op, b=_log(rng, 1, 16), q=rng.randint(2, 40 if tree else 10),
                    v=_log(rng, 1000, 60000), tree=tree)
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128, 256])
    group = rng.choice([v for v in (32, 64, 128) if v <= d])
    heads = dict(hq=hkv * rng.choice([1, 2, 4, 5, 8]), hkv=hkv, d=d, g=group,
                 page=rng.choice([16, 32, 64, 128]))
    if op == "append":
        q = _log(rng, 1, 700)
        return dict(op=op, b=_log(rng, 1, 4 if q > 100 else 64), q=q, len=q + _log(rng, 1, 2000),
                    out=rng.choice(["f32", "bf16"]), **_draw_rope(rng, d), **heads)
    q = rng.randint(2, 64)
    if op == "keep":
        return dict(op=op, b=_log(rng, 1, 48), q=q, len=q + _log(rng, 1, 2000), **heads)
    heads["hq"] = hkv * rng.choice([n for n in (1, 2, 4, 5, 8) if hkv * n <= 40])
    if rng.random() < 0.4:
        return dict(op=op, b=1, q=q, len=_log(rng, 4000, 24000), **heads)
    return dict(op=op, b=_log(rng, 2, 12), q=q, len=q + _log(rng, 1, 2500), **heads)


# ------------------------------------------------------------------ inputs

def _turns(case):
    """Turns per position of each pair of dimensions, and the factor of the rotated vector."""
    r, base, s = case["r"], case["base"], case["s"]
    length, factor = 8192, 1.0
    if case["kind"] == "ntk":
        base *= s ** (r / (r - 2))
    rate = torch.tensor([base ** (-2 * i / r) for i in range(r // 2)], dtype=torch.float64)
    if case["kind"] == "linear":
        rate = rate / s
    elif case["kind"] == "yarn":
        low, high = (r * math.log(length / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32, 1))
        low, high = max(math.floor(low), 0), min(math.ceil(high), r - 1)
        ramp = ((torch.arange(r // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        rate = rate / s * ramp + rate * (1 - ramp)
        factor = 0.1 * math.log(s) + 1
    elif case["kind"] == "bands":
        # whole below a quarter of the length's wavelengths, divided above all of it, mixed between
        mix = ((length * rate / (2 * math.pi) - 1) / (4 - 1)).clamp(0, 1)
        rate = rate / s * (1 - mix) + rate * mix
    return (rate / (2 * math.pi)).to(DEVICE), factor


def _lengths(case):
    """Cached tokens of each sequence, its new ones included: from len down to about half of it."""
    b, q, top = case["b"], case["q"], case["len"]
    return [max(q, top - (i * 7919) % (top // 2 + 1)) for i in range(b)]


def _counts(case):
    """New tokens of each sequence: q, and, from two on, a ragged share of it."""
    q = case["q"]
    return [q if q < 4 else max(2, q - (i * 431) % (q // 2)) for i in range(case["b"])]


def _accepted(counts):
    """Accepted tokens of each sequence, its root included: one to half of the drafts, at most 20."""
    return [1 + (i * 7 + 4) % max(1, min(n // 2, 20)) for i, n in enumerate(counts)]


def _parents(n, rng):
    """A tree of n rows, each behind its parent: row 0 is the root."""
    reach = rng.choice([2, 4, 8])
    return [-1] + [rng.randrange(max(0, (i - 1) // 2 - reach + 1), (i - 1) // 2 + 1) for i in range(1, n)]


def _groups4(x, g):
    """Symmetric 4-bit codes in groups of g along the last axis: (codes -8 .. 7, scales)."""
    v = x.float().unflatten(-1, (-1, g))
    s = v.abs().amax(-1).double().div(7.0).float()
    s = torch.where(s == 0, torch.full_like(s, 1.0 / 7.0), s)
    q = (v.double() / s.double().unsqueeze(-1)).float().round().clamp(-8, 7)
    return q.flatten(-2).to(torch.int64), s


def _nibbles_to_words(q):
    """q [..., 8 n] in storage order -> int32 words, code + 8 in four bits each, LSB first."""
    u = (q + 8).unflatten(-1, (-1, 8))
    w = (u << torch.arange(0, 32, 4, device=q.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _store_order_k(q):
    """Key codes: dimension 32 i + 8 r + e of a head is code e of word r (D / 32) + i."""
    d = q.shape[-1]
    return q.unflatten(-1, (d // 32, 4, 8)).transpose(-3, -2).flatten(-3)


def _store_order_v(q):
    """Value codes: dimension 16 j + c of a head is code c (D / 16) + j of its row."""
    d = q.shape[-1]
    return q.unflatten(-1, (d // 16, 16)).transpose(-2, -1).flatten(-2)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _batch(case, gen):
    """The batch's metadata, and pages in scattered order for every cached token."""
    b, page = case["b"], case["page"]
    lens, counts = _lengths(case), _counts(case)
    per = [-(-v // page) for v in lens]
    width, total = max(per), sum(per)
    pages = total + 3
    order = torch.randperm(pages, generator=gen, device=DEVICE)[:total].to(torch.int32)
    table = torch.zeros(b, width, dtype=torch.int32, device=DEVICE)
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    meta = dict(table=table, lens=_ints(lens), starts=_ints(starts), tokens=starts[-1],
                max_q=max(counts), max_len=max(lens))
    return meta, (pages, case["hkv"], page, case["d"]), counts


def _filled(case, shape, normal):
    """A cache whose every page holds keys and values."""
    keys = normal(*shape)
    keys[..., ::41] *= 4.0
    kq, ks = _groups4(keys, case["g"])
    vq, vs = _groups4(normal(*shape), case["g"])
    return dict(k_codes=_nibbles_to_words(_store_order_k(kq)), k_scales=ks.transpose(-1, -2).contiguous(),
                v_codes=_nibbles_to_words(_store_order_v(vq)), v_scales=vs.transpose(-1, -2).contiguous())


def _prepare_verify(case, seed, gen, normal):
    b, v = case["b"], case["v"]
    counts = _counts(case)
    total = sum(counts)
    rng = random.Random(seed)
    logits = normal(total, v) * 2.5
    draft_logits = logits + normal(total, v) * 0.7
    probs = torch.softmax(logits, -1)
    parents, starts = [], [0]
    for n in counts:
        parents += _parents(n, rng) if case["tree"] else list(range(-1, n - 1))
        starts.append(starts[-1] + n)
    # the draft's row of each token's parent, and how many siblings stand before it
    row, rank, seen = [], [], {}
    for i, n in enumerate(counts):
        for j in range(n):
            at = starts[i] + max(parents[starts[i] + j], 0)
            row.append(at)
            rank.append(seen.get(at, 0) if j else 0)
            seen[at] = rank[-1] + (1 if j else 0)
    row, rank = (torch.tensor(x, device=DEVICE) for x in (row, rank))
    draft = None
    if case["tree"]:  # the candidates of a row: the draft's largest, in order
        best = torch.topk(draft_logits, min(v, max(rank.tolist()) + 1), dim=-1).indices
        tokens = best[row, rank]
    else:
        draft = torch.softmax(draft_logits, -1)
        tokens = torch.multinomial(draft, 1, generator=gen)[:, 0][row]
    return dict(case=case, probs=probs, draft=draft, tokens=tokens.to(torch.int32), parents=_ints(parents),
                starts=_ints(starts), count=b, total=total, most=max(counts),
                uniforms=torch.rand(total, generator=gen, device=DEVICE))


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE)

    if op == "verify":
        return _prepare_verify(case, seed, gen, normal)
    if op == "rotate":
        # queries as the first heads of a fused projection's output, positions up to `far`
        t, h, d = case["t"], case["h"], case["d"]
        qkv = normal(t, h + 2, d) * torch.exp(normal(t, 1, 1))
        qkv = qkv.bfloat16() if case["dtype"] == "bf16" else qkv
        positions = torch.arange(t, device=DEVICE) % 1000 + max(0, case["far"] - 1000)
        state = dict(case=case, x=qkv[:, :h], positions=positions.to(torch.int32))
        state["turns"], state["factor"] = _turns(case)
        return _plan(state)

    meta, shape, counts = _batch(case, gen)
    hq, hkv, d, t = case["hq"], case["hkv"], case["d"], meta["tokens"]
    state = dict(case=case, **meta)
    if op == "append":
        # keys and values as slices of a fused projection's output
        qkv = normal(t, hq + 2 * hkv, d)
        qkv[:, :, ::41] *= 6.0
        qkv = qkv.bfloat16()
        words = torch.zeros(shape[0], hkv, shape[2], d // 8, dtype=torch.int32, device=DEVICE)
        scales = torch.zeros(shape[0], hkv, d // case["g"], shape[2], device=DEVICE)
        state.update(k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], k_codes=words,
                     v_codes=words.clone(), k_scales=scales, v_scales=scales.clone())
        state["turns"], state["factor"] = _turns(case)
        return _plan(state)
    state.update(_filled(case, shape, normal))
    rng = random.Random(seed)
    if op == "keep":
        # accepted rows: the root, then rows behind the places that they move to
        path, accepted = [], _accepted(counts)
        for n, a in zip(counts, accepted):
            path += [0] + sorted(rng.sample(range(a, n), a - 1)) + [-1] * (n - a)
        kept = [0]
        for a in accepted:
            kept.append(kept[-1] + a)
        state.update(path=_ints(path), accepted=_ints(accepted), kept=kept[-1], kept_starts=_ints(kept),
                     kept_lens=state["lens"] - _ints(counts) + _ints(accepted))
        return _plan(state)
    words = -(-meta["max_q"] // 32)
    mask, parents = [], []
    for n in counts:
        tree = _parents(n, rng)
        parents += tree
        bits = []
        for i in range(n):
            bits.append(1 << i | (bits[tree[i]] if i else 0))
        for m in bits:
            mask.append([(m >> 32 * w & 0xFFFFFFFF ^ 0x80000000) - 0x80000000 for w in range(words)])
    state.update(mask=_ints(mask), parents=parents, q=(normal(t, hq, d) * 2.0).bfloat16())
    return _plan(state)


def _plan(state):
    """What a program keeps over its calls: the cache's handle, the rotation's table."""
    if own:
        import mixed_precision_weight_dq_amd as dq
        case = state["case"]
        if "k_codes" in state:
            state["cache"] = dq.Cache4(*(state[n] for n in ("k_codes", "v_codes", "k_scales", "v_scales")))
        if "r" in case:
            scaling = None if case["kind"] == "none" else dict(kind=case["kind"], factor=case["s"],
                                                               length=8192)
            state["rope"] = dq.Rope(case["r"], base=case["base"], interleaved=case["inter"],
                                    scaling=scaling, device=DEVICE)
    return state


# ------------------------------------------------------------- plain forms

def _rotated(x, positions, turns, factor, inter, kind):
    """x [tokens, heads, D] with its first 2 len(turns) dimensions rotated, in dtype kind."""
    r = 2 * turns.shape[0]
    angle = positions.double().unsqueeze(1) * turns
    angle = (angle - angle.round()) * (2 * math.pi)
    c, s = ((f(angle) * factor).to(kind).unsqueeze(1) for f in (torch.cos, torch.sin))
    x = x.to(kind)
    out = x.clone()
    if inter:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        out[..., 0:r:2], out[..., 1:r:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        out[..., :r // 2], out[..., r // 2:r] = a * c - b * s, b * c + a * s
    return out


def _plain_rotate(s):
    out = _rotated(s["x"], s["positions"], s["turns"], s["factor"], s["case"]["inter"], torch.float32)
    return out.to(s["x"].dtype)


def _values(words, scales, g, key):
    """Dequantized rows [..., D] of words [..., P, D / 8] and scales [..., D / g, P]."""
    shifts = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    u = ((words.unsqueeze(-1) >> shifts) & 15).flatten(-2)
    d = u.shape[-1]
    if key:
        u = u.unflatten(-1, (4, d // 32, 8)).transpose(-3, -2).flatten(-3)
    else:
        u = u.unflatten(-1, (16, d // 16)).transpose(-2, -1).flatten(-2)
    return (u.float() - 8.0) * scales.transpose(-1, -2).repeat_interleave(g, -1)


def _places(s, page, tokens, starts, lens):
    """For every token: its sequence, position, page and offset in the page."""
    starts, lens = starts.long(), lens.long()
    t = torch.arange(tokens, device=starts.device)
    seq = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    pos = lens[seq] - (starts[seq + 1] - t)
    return seq, pos, s["table"].long()[seq, pos // page], pos % page


def _read(s, page, off, kind):
    g = s["case"]["g"]
    k = _values(s["k_codes"][page, :, off].unsqueeze(-2), s["k_scales"][page, :, :, off].unsqueeze(-1), g, True)
    v = _values(s["v_codes"][page, :, off].unsqueeze(-2), s["v_scales"][page, :, :, off].unsqueeze(-1), g, False)
    return k.squeeze(-2).to(kind), v.squeeze(-2).to(kind)


def _plain_append(s):
    case = s["case"]
    g = case["g"]
    _, pos, page, off = _places(s, case["page"], s["tokens"], s["starts"], s["lens"])
    # in 64 bits, then rounded to 32: a code next to a border goes by that value
    k = _rotated(s["k"], pos, s["turns"], s["factor"], case["inter"], torch.float64).float()
    kq, ks = _groups4(k, g)
    vq, vs = _groups4(s["v"], g)
    s["k_codes"][page, :, off] = _nibbles_to_words(_store_order_k(kq))
    s["v_codes"][page, :, off] = _nibbles_to_words(_store_order_v(vq))
    s["k_scales"][page, :, :, off] = ks
    s["v_scales"][page, :, :, off] = vs
    return _read(s, page, off, torch.bfloat16 if case["out"] == "bf16" else torch.float32)


def _plain_attention(s):
    case = s["case"]
    hq, hkv, d, g, page = (case[n] for n in ("hq", "hkv", "d", "g", "page"))
    b, width = s["table"].shape
    table, lens = s["table"].long(), s["lens"].long()
    length = width * page

    def rows(codes, scales, key):  # [B, Hkv, L, D], zeros past each sequence's end
        x = _values(codes[table], scales[table], g, key)
        x = x.transpose(1, 2).reshape(b, hkv, length, d)
        return x * (torch.arange(length, device=x.device) < lens.unsqueeze(1))[:, None, :, None]

    starts = s["starts"].long()
    seq, _, _, _ = _places(s, page, s["tokens"], s["starts"], s["lens"])
    at = torch.arange(s["tokens"], device=seq.device) - starts[seq]
    q = torch.zeros(b, s["max_q"], hq, d, device=seq.device)
    q[seq, at] = s["q"].float()
    # which positions a token sees: the context, and the new ones of its bits
    new = torch.arange(length, device=seq.device) - (lens - (starts[1:] - starts[:-1])).unsqueeze(1)
    bits = s["mask"].long()[:, :, None] >> torch.arange(32, device=seq.device) & 1
    bits = torch.nn.functional.pad(bits.flatten(1), (0, 1)).bool()
    inside = torch.where((new >= 0) & (new < bits.shape[1] - 1), new, bits.shape[1] - 1)
    sees = torch.zeros(b, s["max_q"], length, dtype=torch.bool, device=seq.device)
    sees[seq, at] = torch.gather(bits, 1, inside[seq]) | (new < 0)[seq]
    sees &= (torch.arange(length, device=seq.device) < lens.unsqueeze(1)).unsqueeze(1)

    per = hq // hkv
    q = q.view(b, s["max_q"], hkv, per, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    logits = torch.matmul(q, rows(s["k_codes"], s["k_scales"], True).transpose(-1, -2).contiguous()) * d ** -0.5
    logits = logits.view(b, hkv, per, s["max_q"], length)
    logits.masked_fill_(~sees[:, None, None], -torch.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(logits.sub_(top))
    o = torch.matmul(p.view(b, hkv, -1, length), rows(s["v_codes"], s["v_scales"], False))
    o = o / p.sum(-1).view(b, hkv, -1, 1).clamp(min=1e-38)
    o = o.view(b, hkv, per, s["max_q"], d).permute(0, 3, 1, 2, 4).reshape(b, -1, hq, d)
    return o[seq, at].bfloat16()


def _plain_verify(s):
    b, total = s["count"], s["total"]
    probs, draft, tokens, u = s["probs"], s["draft"], s["tokens"].long(), s["uniforms"].double()
    starts, parents = s["starts"].long(), s["parents"].long()
    first, n = starts[:-1], starts[1:] - starts[:-1]
    rows = torch.arange(b, device=first.device)
    cur = torch.zeros_like(first)                       # the last accepted row of each sequence
    rest = torch.ones(b, dtype=torch.float64, device=first.device)
    refused = torch.zeros(b, dtype=torch.bool, device=first.device)  # by the draft's probabilities
    at = torch.ones_like(first)                         # accepted so far
    path = torch.full((total,), -1, dtype=torch.int32, device=first.device)
    path[first] = 0
    dead = torch.zeros(b, probs.shape[1], dtype=torch.bool, device=first.device)  # refused candidates
    for i in range(1, s["most"]):
        live = i < n
        row = (first + i).clamp(max=total - 1)
        token = tokens[row]
        mine = live & (parents[row] == cur) & ~refused
        p = probs[first + cur, token].double()
        if draft is None:
            p = torch.where(dead[rows, token], 0.0, p)
            take = mine & (u[row] * rest < p)
        else:
            take = mine & (u[row] * draft[first + cur, token].double() < p)
        lost = mine & ~take
        if draft is None:
            rest = torch.where(take, 1.0, torch.where(lost, rest - p, rest))
            dead = dead & ~take.unsqueeze(1)
            dead[rows, token] = torch.where(lost, True, dead[rows, token])
        else:
            refused |= lost
        path[torch.where(take, first + at, 0)] = torch.where(take, i, path[0]).to(torch.int32)
        cur = torch.where(take, i, cur)
        at = at + take
    left = probs[first + cur].double()
    if draft is None:
        left = left.masked_fill(dead, 0.0)
    else:
        left = torch.where(refused.unsqueeze(1), (left - draft[first + cur].double()).clamp(min=0), left)
    upto = left.cumsum(-1)
    last = (upto <= (u[first] * upto[:, -1]).unsqueeze(1)).sum(-1)
    return path, at.to(torch.int32), last.to(torch.int32)


def _plain_keep(s):
    case = s["case"]
    seq, pos, page, off = _places(s, case["page"], s["kept"], s["kept_starts"], s["kept_lens"])
    starts = s["starts"].long()
    j = torch.arange(s["kept"], device=seq.device) - s["kept_starts"].long()[seq]
    old = s["lens"].long()[seq] - (starts[seq + 1] - starts[seq]) + s["path"].long()[starts[seq] + j]
    old_page, old_off = s["table"].long()[seq, old // case["page"]], old % case["page"]
    for name in ("k_codes", "v_codes"):
        s[name][page, :, off] = s[name][old_page, :, old_off]
    for name in ("k_scales", "v_scales"):
        s[name][page, :, :, off] = s[name][old_page, :, :, old_off]
    return _read(s, page, off, torch.float32)


# --------------------------------------------------------------------- run

def _own(s):
    import mixed_precision_weight_dq_amd as dq
    case = s["case"]
    op = case["op"]
    if op == "rotate":
        return dq.rotate(s["rope"], s["x"], s["positions"])
    if op == "append":
        dq.cache4_append(s["cache"], s["k"], s["v"], s["starts"], s["lens"], s["table"], rope=s["rope"])
        return dq.cache4_read(s["cache"], s["tokens"], s["starts"], s["lens"], s["table"],
                              dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    if op == "attention":
        return dq.cache4_tree_attention(s["cache"], s["q"], s["starts"], s["lens"], s["table"], s["mask"],
                                        max_q=s["max_q"], max_len=s["max_len"])
    if op == "verify":
        return dq.verify_drafts(s["probs"], s["tokens"], s["parents"], s["starts"], s["uniforms"],
                                draft_probs=s["draft"])
    dq.cache4_keep(s["cache"], s["starts"], s["lens"], s["table"], s["path"], s["accepted"])
    return dq.cache4_read(s["cache"], s["kept"], s["kept_starts"], s["kept_lens"], s["table"])


def run(state):
    if own:
        return _own(state)
    plain = {"rotate": _plain_rotate, "append": _plain_append, "attention": _plain_attention,
             "verify": _plain_verify, "keep": _plain_keep}
    return plain[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "rotate":
        n = case["t"] * case["h"]
        size = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=2 * n * case["d"] * size + 4 * case["t"], flops=3 * n * case["r"])
    counts = _counts(case)
    new = sum(counts)
    if op == "verify":
        # one row of the target's probabilities, for a chain often one of the draft's beside it
        rows = case["b"] * (1 if case["tree"] else 2)
        return dict(bytes=4 * rows * case["v"] + 24 * new, flops=2 * rows * case["v"])
    hq, hkv, d, g = case["hq"], case["hkv"], case["d"], case["g"]
    held = hkv * (d + 8 * (d // g))  # bytes of one token's codes and scales, keys and values
    if op == "append":
        size = 2 if case["out"] == "bf16" else 4
        return dict(bytes=new * (2 * hkv * d * (2 + size) + 2 * held),
                    flops=new * hkv * (8 * d + 3 * case["r"]))
    if op == "keep":
        # the accepted: read, written, read again, and given out in 32 bits
        kept = sum(_accepted(counts))
        return dict(bytes=kept * (3 * held + 8 * hkv * d), flops=kept * 2 * hkv * d)
    lens = _lengths(case)
    pairs = sum(q * (n - q + 1) for q, n in zip(counts, lens))
    return dict(bytes=sum(lens) * held + 2 * new * hq * d * 2 + 4 * new * -(-max(counts) // 32),
                flops=4 * pairs * hq * d)


# ----------------------------------------------------------- in 64 bits

def _exact_rates(case):
    """Radians per position of each pair, from the definitions, and the factor."""
    r, b, s, length = case["r"], case["base"], case["s"], 8192.0
    out, factor = [], 1.0
    for i in range(r // 2):
        w = math.exp(-2 * i / r * math.log(b))
        if case["kind"] == "linear":
            w /= s
        if case["kind"] == "ntk":
            w = math.exp(-2 * i / r * (math.log(b) + r / (r - 2) * math.log(s)))
        if case["kind"] == "yarn":
            # the pairs that turn 32 times and once over the length bound the ramp
            pair = [r * math.log(length / (2 * math.pi * n)) / (2 * math.log(b)) for n in (32, 1)]
            lo, hi = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), r - 1)
            part = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            w = w * (1 - part) + w / s * part
            factor = 1 + math.log(s) / 10
        if case["kind"] == "bands":
            wave = 2 * math.pi / w
            if wave > length:
                w /= s
            elif wave > length / 4:
                part = (length / wave - 1) / 3
                w = (1 - part) * w / s + part * w
        out.append(w)
    return torch.tensor(out, dtype=torch.float64, device=DEVICE), factor


def _exact_rotated(case, x, positions):
    w, factor = _exact_rates(case)
    r = case["r"]
    turn = torch.polar(torch.full((), factor, dtype=torch.float64, device=DEVICE),
                       positions.double()[:, None] * w)
    x = x.double()
    pair = x[..., :r].unflatten(-1, (-1, 2) if case["inter"] else (2, -1))
    pair = pair if case["inter"] else pair.transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None])
    z = z if case["inter"] else z.transpose(-1, -2)
    return torch.cat([z.flatten(-2), x[..., r:]], -1)


def _exact_verify(s):
    """The rule for one sequence at a time, on the host."""
    starts, parents, tokens = (s[n].tolist() for n in ("starts", "parents", "tokens"))
    u = s["uniforms"].double().tolist()
    path, accepted, last = [-1] * s["total"], [], []
    for b in range(s["count"]):
        f, n = starts[b], starts[b + 1] - starts[b]
        cur, at = 0, 1
        path[f] = 0
        while True:
            p = s["probs"][f + cur].double()
            q = None if s["draft"] is None else s["draft"][f + cur].double()
            went = None
            mass = 1.0
            for c in [i for i in range(cur + 1, n) if parents[f + i] == cur]:
                tok = tokens[f + c]
                if u[f + c] * (mass if q is None else float(q[tok])) < float(p[tok]):
                    went = c
                    break
                if q is not None:
                    p = torch.relu(p - q)
                    break
                mass -= float(p[tok])
                p[tok] = 0.0
            if went is None:
                break
            cur = went
            path[f + at] = cur
            at += 1
        accepted.append(at)
        total = torch.cumsum(p, 0)
        last.append(int(torch.searchsorted(total, u[f] * total[-1], right=True)))
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (path, accepted, last))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotate":
        return _exact_rotated(case, s["x"], s["positions"])
    if op == "verify":
        return _exact_verify(s)
    d, g, hq, hkv, page = (case[n] for n in ("d", "g", "hq", "hkv", "page"))
    lens, counts = _lengths(case), _counts(case)
    dims = torch.arange(d, device=DEVICE)
    if op == "append":
        pos = torch.cat([torch.arange(n - q, n) for n, q in zip(lens, counts)]).to(DEVICE)
        out = []
        for x in (_exact_rotated(case, s["k"], pos).float().double(), s["v"].double()):
            # the stored scale is a 32-bit number: it is part of the format
            scale = torch.stack([x[..., i:i + g].abs().amax(-1) for i in range(0, d, g)], -1) / 7.0
            scale = scale.float().double()[..., dims // g]
            out.append(torch.clamp(torch.round((x / scale).float().double()), -8, 7) * scale)
        return tuple(out)
    # where dimension x of a head lies in its row of 4-bit codes
    at_k = (((dims % 32) // 8) * (d // 32) + dims // 32) * 8 + dims % 8
    at_v = (dims % 16) * (d // 16) + dims // 16

    def entries(i, t):  # keys and values of positions t of sequence i, [len(t), Hkv, D]
        pages, off = s["table"][i].long()[t // page], t % page
        kv = []
        for name, at in (("k", at_k), ("v", at_v)):
            word = s[name + "_codes"][pages, :, off].long()[..., at // 8]
            code = ((word >> (4 * (at % 8))) & 15).double() - 8.0
            kv.append(code * s[name + "_scales"][pages, :, :, off].double()[..., dims // g])
        return kv

    if op == "keep":
        path, starts, accepted = (s[n].tolist() for n in ("path", "starts", "accepted"))
        both = [entries(i, torch.tensor([n - q + r for r in path[f:f + a]], device=DEVICE))
                for i, (n, q, f, a) in enumerate(zip(lens, counts, starts, accepted))]
        return torch.cat([k for k, _ in both]), torch.cat([v for _, v in both])
    out = torch.empty(s["tokens"], hq, d, dtype=torch.float64, device=DEVICE)
    first = 0
    for i, (n, q) in enumerate(zip(lens, counts)):
        k, v = entries(i, torch.arange(n, device=DEVICE))
        hidden = torch.zeros(q, n, dtype=torch.bool)
        hidden[:, n - q:] = True
        for r in range(q):
            c = r
            while c >= 0:
                hidden[r, n - q + c] = False
                c = s["parents"][first + c]
        hidden = hidden.to(DEVICE)
        for h in range(hq):
            a = s["q"][first:first + q, h].double() @ k[:, h // (hq // hkv)].t() / math.sqrt(d)
            a = a.masked_fill(hidden, -math.inf)
            out[first:first + q, h] = torch.softmax(a, -1) @ v[:, h // (hq // hkv)]
        first += q
    return out
