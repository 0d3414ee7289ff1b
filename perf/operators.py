"""Cases that measure the 8-bit activation and 4-bit cache operators.

A quantized serving step holds three kinds of tensors in few bits: the weights
(b-bit codes, packed), the activations that meet them (int8 codes, one scale
per token) and the key/value cache (4-bit codes in pages, one scale per group
of a head's dimensions).  The operators here are the ones around the last two:

* ``tokens``    -- quantize activations to int8, one scale per token;
* ``product``   -- int8 activations times packed b-bit weights, exact integer
                   sums, scaled per token and per channel;
* ``append``    -- quantize new keys and values into the paged 4-bit cache (and
                   read them back, which is how the stored values are seen);
* ``attention`` -- causal attention of new queries over that cache.

``run`` computes each in elementary torch operations, or, where ``own`` is
true, through the package.  Shapes: 4096-, 5120-, 8192-wide layers with 17408-
and 28672-wide projections, heads of 64 or 128, eight or fewer kv heads.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token's hidden state on its way into a projection
        dict(name="tokens-1x4096", op="tokens", m=1, k=4096, dtype="bf16"),
        # a prompt's hidden states
        dict(name="tokens-2048x8192", op="tokens", m=2048, k=8192, dtype="bf16"),
        # decode of one sequence: a square projection at 4 bits
        dict(name="product-1x4096x4096-b4", op="product", m=1, n=4096, k=4096, bits=4, asym=False,
             out="f32"),
        # decode of a batch: a wide projection at 6 bits
        dict(name="product-16x28672x8192-b6", op="product", m=16, n=28672, k=8192, bits=6,
             asym=False, out="f32"),
        # a prompt through a square projection at 8 bits
        dict(name="product-2048x8192x8192-b8", op="product", m=2048, n=8192, k=8192, bits=8,
             asym=False, out="f32"),
        # a short prompt of odd length, zero points, 5 bits, bf16 out
        dict(name="product-333x17408x5120-b5z", op="product", m=333, n=17408, k=5120, bits=5,
             asym=True, out="bf16"),
        # a decode step's new tokens of 32 sequences into the cache
        dict(name="append-32x1", op="append", b=32, q=1, len=2000, hq=32, hkv=8, d=128, g=32,
             page=64, out="f32"),
        # prompts into the cache
        dict(name="append-3x2500", op="append", b=3, q=2500, len=2900, hq=64, hkv=8, d=128, g=64,
             page=64, out="bf16"),
        # decode of one long sequence: few rows, a long axis
        dict(name="attention-1x1-65000", op="attention", b=1, q=1, len=65000, hq=32, hkv=8, d=128,
             g=32, page=64),
        # decode of a ragged batch
        dict(name="attention-40x1-6000", op="attention", b=40, q=1, len=6000, hq=40, hkv=8, d=128,
             g=32, page=64),
        # drafted tokens verified together, narrow heads, small pages
        dict(name="attention-8x5-1100", op="attention", b=8, q=5, len=1100, hq=16, hkv=4, d=64,
             g=64, page=16),
        # a piece of a prompt over what is cached already
        dict(name="attention-2x1000-6000", op="attention", b=2, q=1000, len=6000, hq=32, hkv=8,
             d=128, g=32, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tokens", "product", "product", "append", "attention", "attention"])
    if op == "tokens":
        return dict(op=op, m=_log(rng, 1, 1000), k=_log(rng, 32, 8000),
                    dtype=rng.choice(["bf16", "f32"]))
    if op == "product":
        m = _log(rng, 1, 1200)
        k = rng.choice([1024, 4096, 5120, 8192, _log(rng, 33, 9000)])
        return dict(op=op, m=m, n=_log(rng, 64, 12000), k=k, bits=rng.randint(2, 8),
                    asym=rng.random() < 0.4, out=rng.choice(["f32", "bf16"]))
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128, 256])
    group = rng.choice([v for v in (32, 64, 128) if v <= d])
    heads = dict(hq=hkv * rng.choice([1, 2, 4, 5, 8]), hkv=hkv, d=d, g=group,
                 page=rng.choice([16, 32, 64, 128]))
    if op == "append":
        q = _log(rng, 1, 700)
        return dict(op=op, b=_log(rng, 1, 4 if q > 100 else 64), q=q, len=q + _log(rng, 1, 2000),
                    out=rng.choice(["f32", "bf16"]), **heads)
    kind = rng.choice(["long", "batch", "draft", "prompt"])
    if kind == "long":
        return dict(op=op, b=rng.randint(1, 2), q=1, len=_log(rng, 8000, 32000), **heads)
    if kind == "batch":
        return dict(op=op, b=_log(rng, 3, 24), q=1, len=_log(rng, 20, 4000), **heads)
    if kind == "draft":
        return dict(op=op, b=_log(rng, 1, 16), q=rng.randint(2, 9), len=_log(rng, 20, 3000), **heads)
    q = _log(rng, 20, 400)
    return dict(op=op, b=rng.randint(1, 2), q=q, len=q + _log(rng, 1, 2000), **heads)


# ------------------------------------------------------------------ inputs

def _pad128(k):
    return -(-k // 128) * 128


def _row_words(k, bits):
    return -(-(-(-k * bits // 8)) // 128) * 32


def _pack(u, bits):
    """Codes u [N, K] (int64) as one LSB-first bit stream per row, rows padded to 128 bytes."""
    n, k = u.shape
    chunks = -(-k // 32)
    rw = _row_words(k, bits)
    u = torch.nn.functional.pad(u, (0, chunks * 32 - k)).view(n, chunks, 32)
    words = torch.zeros(n, chunks, bits + 1, dtype=torch.int64, device=u.device)
    for j in range(32):
        v = u[:, :, j] << (j * bits % 32)
        words[:, :, j * bits // 32] |= v & 0xFFFFFFFF
        words[:, :, j * bits // 32 + 1] |= v >> 32
    flat = words[:, :, :bits].reshape(n, chunks * bits)
    out = torch.zeros(n, rw, dtype=torch.int64, device=u.device)
    out[:, :min(rw, flat.shape[1])] = flat[:, :rw]
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32)


def _lengths(case):
    """Cached tokens of each sequence, its new ones included: from len down to about half of it."""
    b, q, top = case["b"], case["q"], case["len"]
    return [max(q, top - (i * 7919) % (top // 2 + 1)) for i in range(b)]


def _queries(case):
    """New tokens of each sequence: q, and for prompts a ragged share of it."""
    q = case["q"]
    return [q if q < 16 else max(1, q - (i * 431) % (q // 2)) for i in range(case["b"])]


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


def _cache(case, gen):
    """The batch's metadata, and pages (in scattered order) that hold every cached token."""
    b, hkv, d, g, page = (case[n] for n in ("b", "hkv", "d", "g", "page"))
    lens, qs = _lengths(case), _queries(case)
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
    for n in qs:
        starts.append(starts[-1] + n)
    meta = dict(table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEVICE),
                starts=torch.tensor(starts, dtype=torch.int32, device=DEVICE),
                tokens=starts[-1], max_q=max(qs), max_len=max(lens))
    shape = (pages, hkv, page, d)
    return meta, shape, g


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEVICE)

    if op in ("tokens", "product"):
        m, k = case["m"], case["k"]
        x = normal(m, k) * torch.exp(normal(m, 1))
        x[:, ::97] *= 12.0  # the few channels that run hot
        if op == "tokens":
            return dict(case=case, x=x.bfloat16() if case["dtype"] == "bf16" else x)
        n, bits = case["n"], case["bits"]
        codes, scale, sums = _quantize_tokens(x.bfloat16())
        w = normal(n, k)
        top = 2 ** bits - 1
        if case["asym"]:
            w += 0.5
            lo, hi = w.amin(1, keepdim=True).clamp(max=0), w.amax(1, keepdim=True).clamp(min=0)
            s = (hi - lo) / top
            z = (-lo / s).round().clamp(0, top)
            u = ((w / s).round() + z).clamp(0, top).to(torch.int64)
            zeros = z[:, 0].to(torch.int32)
        else:
            s = w.abs().amax(1, keepdim=True) / (2 ** (bits - 1) - 1)
            u = (w / s).round().to(torch.int64) + 2 ** (bits - 1)
            zeros = None
        return dict(case=case, codes=codes, x_scale=scale, x_sums=sums, packed=_pack(u, bits),
                    w_scale=(s[:, 0] * 0.02).contiguous(), zeros=zeros)

    meta, shape, g = _cache(case, gen)
    pages, hkv, page, d = shape
    hq, t = case["hq"], meta["tokens"]
    state = dict(case=case, **meta)
    if op == "append":
        # keys and values as slices of a fused projection's output
        qkv = normal(t, hq + 2 * hkv, d)
        qkv[:, :, ::41] *= 6.0
        qkv = qkv.bfloat16()
        words = torch.zeros(pages, hkv, page, d // 8, dtype=torch.int32, device=DEVICE)
        scales = torch.zeros(pages, hkv, d // g, page, device=DEVICE)
        state.update(k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], k_codes=words,
                     v_codes=words.clone(), k_scales=scales, v_scales=scales.clone())
        return state
    keys = normal(*shape)
    keys[..., ::41] *= 4.0
    kq, ks = _groups4(keys, g)
    state["k_codes"] = _nibbles_to_words(_store_order_k(kq))
    state["k_scales"] = ks.transpose(-1, -2).contiguous()
    del keys, kq, ks
    vq, vs = _groups4(normal(*shape), g)
    state["v_codes"] = _nibbles_to_words(_store_order_v(vq))
    state["v_scales"] = vs.transpose(-1, -2).contiguous()
    state["q"] = (normal(t, hq, d) * 2.0).bfloat16()
    return state


# ------------------------------------------------------------- plain forms

def _quantize_tokens(x):
    m, k = x.shape
    v = x.float()
    top = v.abs().amax(1)
    scale = (torch.where(top == 0, torch.ones_like(top), top).double() / 127.0).float()
    q = (v.double() / scale.double().unsqueeze(1)).float().round().clamp(-128, 127)
    codes = torch.zeros(m, _pad128(k), dtype=torch.int8, device=x.device)
    codes[:, :k] = q.to(torch.int8)
    return codes, scale, codes.sum(1, dtype=torch.int32)


def _unpack(packed, k, bits):
    """The codes of packed rows as float32 [N, K]."""
    at = torch.arange(k, device=packed.device) * bits
    word, off = at // 32, (at % 32).to(torch.int32)
    low = (packed[:, word] >> off) & ((1 << torch.clamp(32 - off, max=bits)) - 1)
    spill = torch.clamp(off + bits - 32, min=0)
    high = packed[:, torch.clamp(word + 1, max=packed.shape[1] - 1)] & ((1 << spill) - 1)
    return (low | (high << (bits - spill))).float()


def _plain_product(s):
    case = s["case"]
    q = _unpack(s["packed"], case["k"], case["bits"])
    q -= 2.0 ** (case["bits"] - 1) if s["zeros"] is None else s["zeros"].float().unsqueeze(1)
    y = s["codes"][:, :case["k"]].float() @ q.t()
    y = y * s["x_scale"].unsqueeze(1) * s["w_scale"]
    return y.bfloat16() if case["out"] == "bf16" else y


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


def _places(s, page):
    """For every new token: its sequence, position, page and offset in the page."""
    starts, lens = s["starts"].long(), s["lens"].long()
    t = torch.arange(s["tokens"], device=starts.device)
    seq = torch.searchsorted(starts[1:].contiguous(), t, right=True)
    pos = lens[seq] - (starts[seq + 1] - t)
    return seq, pos, s["table"].long()[seq, pos // page], pos % page


def _plain_append(s):
    case = s["case"]
    g = case["g"]
    _, _, page, off = _places(s, case["page"])
    kq, ks = _groups4(s["k"], g)
    vq, vs = _groups4(s["v"], g)
    s["k_codes"][page, :, off] = _nibbles_to_words(_store_order_k(kq))
    s["v_codes"][page, :, off] = _nibbles_to_words(_store_order_v(vq))
    s["k_scales"][page, :, :, off] = ks
    s["v_scales"][page, :, :, off] = vs
    kind = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    k = _values(s["k_codes"][page, :, off].unsqueeze(-2),
                s["k_scales"][page, :, :, off].unsqueeze(-1), g, True)
    v = _values(s["v_codes"][page, :, off].unsqueeze(-2),
                s["v_scales"][page, :, :, off].unsqueeze(-1), g, False)
    return k.squeeze(-2).to(kind), v.squeeze(-2).to(kind)


def _plain_attention(s):
    case = s["case"]
    hq, hkv, d, g, page = (case[n] for n in ("hq", "hkv", "d", "g", "page"))
    b, width = s["table"].shape
    table = s["table"].long()

    def rows(codes, scales, key):  # [B, Hkv, L, D], zeros past each sequence's end
        x = _values(codes[table], scales[table], g, key)
        x = x.transpose(1, 2).reshape(b, hkv, width * page, d)
        live = torch.arange(width * page, device=x.device) < s["lens"].unsqueeze(1)
        return x * live[:, None, :, None]

    seq, pos, _, _ = _places(s, page)
    at = torch.arange(s["tokens"], device=seq.device) - s["starts"].long()[seq]
    q = torch.zeros(b, s["max_q"], hq, d, device=seq.device)
    q[seq, at] = s["q"].float()
    last = torch.full((b, s["max_q"]), -1, dtype=torch.long, device=seq.device)
    last[seq, at] = pos
    q = q.view(b, s["max_q"], hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    logits = torch.matmul(q, rows(s["k_codes"], s["k_scales"], True).transpose(-1, -2)) * d ** -0.5
    hidden = torch.arange(width * page, device=seq.device) > last.unsqueeze(-1)
    hidden = hidden[:, None, None].expand(b, hkv, hq // hkv, -1, -1).reshape(logits.shape)
    logits.masked_fill_(hidden, -torch.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(logits.sub_(top))
    o = torch.matmul(p, rows(s["v_codes"], s["v_scales"], False))
    o = o / p.sum(-1, keepdim=True).clamp(min=1e-38)
    o = o.view(b, hkv, hq // hkv, s["max_q"], d).permute(0, 3, 1, 2, 4).reshape(b, -1, hq, d)
    return o[seq, at].bfloat16()


# --------------------------------------------------------------------- run

def _own(s):
    import mixed_precision_weight_dq_amd as dq
    case = s["case"]
    if case["op"] == "tokens":
        return dq.quantize_tokens(s["x"])
    if case["op"] == "product":
        product = dq.gemv_i8 if case["m"] <= 16 else dq.gemm_i8
        return product(s["codes"], s["x_scale"], s["x_sums"], s["packed"], s["w_scale"], case["k"],
                       case["bits"], zeros=s["zeros"],
                       dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    cache = dq.Cache4(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
    if case["op"] == "append":
        dq.cache4_append(cache, s["k"], s["v"], s["starts"], s["lens"], s["table"])
        return dq.cache4_read(cache, s["tokens"], s["starts"], s["lens"], s["table"],
                              dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
    return dq.cache4_attention(cache, s["q"], s["starts"], s["lens"], s["table"],
                               max_q=s["max_q"], max_len=s["max_len"])


def run(state):
    if own:
        return _own(state)
    plain = {"tokens": lambda s: _quantize_tokens(s["x"]), "product": _plain_product,
             "append": _plain_append, "attention": _plain_attention}
    return plain[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op == "tokens":
        m, k = case["m"], case["k"]
        return dict(bytes=m * (k * (2 if case["dtype"] == "bf16" else 4) + _pad128(k) + 8),
                    flops=3 * m * k)
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        size = 2 if case["out"] == "bf16" else 4
        return dict(bytes=m * (_pad128(k) + 8) + n * (4 * _row_words(k, case["bits"]) + 4
                                                      + (4 if case["asym"] else 0)) + m * n * size,
                    flops=2 * m * n * k)
    hq, hkv, d, g = case["hq"], case["hkv"], case["d"], case["g"]
    held = hkv * (d + 8 * (d // g))  # bytes of one token's codes and scales, keys and values
    lens, qs = _lengths(case), _queries(case)
    new = sum(qs)
    if op == "append":
        size = 2 if case["out"] == "bf16" else 4
        return dict(bytes=new * (2 * hkv * d * (2 + size) + 2 * held), flops=8 * new * hkv * d)
    pairs = sum(q * n - q * (q - 1) // 2 for q, n in zip(qs, lens))
    return dict(bytes=sum(lens) * held + 2 * new * hq * d * 2, flops=4 * pairs * hq * d)


# ----------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tokens":
        return None, s["x"].double().abs().max(dim=1).values / 127.0, None
    if op == "product":
        bits, k = case["bits"], case["k"]
        words = s["packed"].to(torch.int64) & 0xFFFFFFFF
        w = torch.empty(words.shape[0], k, dtype=torch.float64, device=words.device)
        for j in range(min(32, k)):  # code j of every 32-code chunk
            first, off = divmod(j * bits, 32)
            n = len(range(j, k, 32))
            u = words[:, first::bits][:, :n] >> off
            if off + bits > 32:
                u = u | words[:, first + 1::bits][:, :n] << (32 - off)
            w[:, j::32] = (u & (2 ** bits - 1)).double()
        w -= float(2 ** (bits - 1)) if s["zeros"] is None else s["zeros"].double()[:, None]
        w *= s["w_scale"].double()[:, None]
        x = s["codes"][:, :k].double() * s["x_scale"].double()[:, None]
        return torch.mm(x, w.t())
    d, g, hq, hkv, page = (case[n] for n in ("d", "g", "hq", "hkv", "page"))
    dims = torch.arange(d, device=DEVICE)
    if op == "append":
        out = []
        for x in (s["k"], s["v"]):
            x = x.double()
            # the stored scale is a 32-bit number: it is part of the format
            scale = torch.stack([x[..., i:i + g].abs().amax(-1) for i in range(0, d, g)], -1) / 7.0
            scale = scale.float().double()[..., dims // g]
            out.append(torch.clamp(torch.round((x / scale).float().double()), -8, 7) * scale)
        return tuple(out)
    # where dimension x of a head lies in its row of 4-bit codes
    at_k = (((dims % 32) // 8) * (d // 32) + dims // 32) * 8 + dims % 8
    at_v = (dims % 16) * (d // 16) + dims // 16
    out = torch.empty(s["tokens"], hq, d, dtype=torch.float64, device=DEVICE)
    for i, (n, q) in enumerate(zip(_lengths(case), _queries(case))):
        t = torch.arange(n, device=DEVICE)
        pages, off = s["table"][i].long()[t // page], t % page
        kv = []
        for name, at in (("k", at_k), ("v", at_v)):
            word = s[name + "_codes"][pages, :, off].long()[..., at // 8]
            code = ((word >> (4 * (at % 8))) & 15).double() - 8.0
            kv.append(code * s[name + "_scales"][pages, :, :, off].double()[..., dims // g])
        first = int(s["starts"][i])
        for h in range(hq):
            k, v = kv[0][:, h // (hq // hkv)], kv[1][:, h // (hq // hkv)]
            a = s["q"][first:first + q, h].double() @ k.t() / math.sqrt(d)
            rows = torch.arange(n - q, n, device=DEVICE)
            a = a.masked_fill(t[None, :] > rows[:, None], -math.inf)
            out[first:first + q, h] = torch.softmax(a, -1) @ v
    return out
