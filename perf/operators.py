"""The serving operators around the index branch, as cases to measure.

A layer of block-sparse attention takes four steps for a chunk of new tokens:
the cache append (rotate the new query and key rows, write keys and values to
their pages, encode the index branch's rows), the block scores with their top
blocks (which bench.py measures), and the attention over the selected blocks;
layers without an index branch attend to the whole cache or the whole prompt.
The cases here are the append, the attention of new tokens over a paged cache,
the attention of whole packed prompts and the attention over selected blocks.

``run`` computes an operator in elementary torch operations where ``own`` is
false, and through the package's entry points where it is true.
"""
import math
import random

import torch

own = False

P = 128            # tokens per block, which is a page
D = 128            # head dimension
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
# op        append | paged | prompt | selected
# B, q_lo, q_hi, ctx_lo, ctx_hi
#           requests; new tokens and earlier tokens of each are drawn from
#           these ranges (over their logarithm) by a generator of the case's
#           own ("lengths"), so the sizes do not depend on the seed
# Hq, Hkv   query and key/value heads; layout of the cache; mode 3 is causal
# k         selected blocks per token; index: the append's index branch
#           ("same", "e4m3", "i8", "mxfp4", "none"), Hi its query heads
# rot, pairs  rotated elements of a head and how they pair up


def _attn(name, op, B, q, ctx, Hq, Hkv, layout, dtype, mode=3, k=0, lengths=1):
    return {"name": name, "op": op, "B": B, "q_lo": q[0], "q_hi": q[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "Hq": Hq, "Hkv": Hkv, "layout": layout, "dtype": dtype,
            "mode": mode, "k": k, "lengths": lengths}


def _app(name, B, q, ctx, Hq, Hkv, Hi, layout, dtype, index, rot, pairs, lengths=1):
    return {"name": name, "op": "append", "B": B, "q_lo": q[0], "q_hi": q[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "Hq": Hq, "Hkv": Hkv, "Hi": Hi, "layout": layout, "dtype": dtype,
            "index": index, "rot": rot, "pairs": pairs, "lengths": lengths}


def listed():
    return [
        # one decode step of a batch of 64: one new token each, the index
        # branch in the model's own type
        _app("append_decode_bf16", 64, (1, 1), (1, 4095), 32, 4, 4, "BBND", "bf16", "same", 128,
             "halves"),
        # four prompts' chunks in one batch, half of each head rotated, fp8
        # index rows
        _app("append_prefill_e4m3", 4, (1000, 8192), (0, 4096), 64, 8, 8, "BBND", "bf16", "e4m3",
             64, "halves"),
        # a long chunk whose index branch is MXFP4, interleaved pairs
        _app("append_chunk_mxfp4", 1, (4096, 4096), (8191, 8191), 32, 4, 16, "BNBD", "f16",
             "mxfp4", 128, "interleaved"),
        # a speculative step of a small batch with int8 index keys
        _app("append_spec_i8", 7, (2, 6), (1, 3000), 16, 1, 16, "BNBD", "f16", "i8", 128,
             "halves"),
        # the smallest chunk: one request of 32 new tokens in two blocks
        _attn("paged_tiny_f16", "paged", 1, (32, 32), (224, 224), 8, 1, "BBND", "f16"),
        # a decode batch over contexts of every length
        _attn("paged_decode_bf16", "paged", 64, (1, 1), (1, 8191), 64, 8, "BBND", "bf16"),
        # a scheduler's mixed batch: decode and speculative tokens beside chunks
        _attn("paged_mixed_f16", "paged", 9, (1, 700), (1, 6000), 32, 4, "BNBD", "f16"),
        # a chunk of a long prompt over its earlier tokens
        _attn("paged_chunk_bf16", "paged", 1, (2048, 2048), (30720, 30720), 32, 4, "BBND", "bf16"),
        # whole prompts of very different lengths, packed
        _attn("prompt_packed_bf16", "prompt", 5, (150, 8192), (0, 0), 32, 4, "TND", "bf16"),
        # short prompts, an odd group of heads
        _attn("prompt_short_f16", "prompt", 6, (1, 300), (0, 0), 12, 4, "TND", "f16"),
        # decode over 16 selected blocks of long contexts
        _attn("selected_decode_bf16", "selected", 64, (1, 1), (1, 32767), 32, 4, "BBND", "bf16",
              k=16),
        # a chunk of a long prompt, each token over its own 16 blocks
        _attn("selected_chunk_bf16", "selected", 1, (4096, 4096), (28673, 28673), 32, 4, "BBND",
              "bf16", k=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 1)),
                                                          math.log(max(hi, 1))))))))


def draw(rng):
    op = rng.choice(["append", "append", "paged", "paged", "prompt", "selected", "selected"])
    dtype = rng.choice(["bf16", "f16"])
    layout = "TND" if op == "prompt" else rng.choice(["BBND", "BNBD"])
    Hq, Hkv = rng.choice([(8, 1), (16, 1), (32, 4), (64, 8), (12, 4), (10, 2), (8, 8)])
    lengths = rng.randrange(1 << 20)
    long = rng.random() < 0.5
    if op == "append":
        B = _log(rng, 1, 8) if long else _log(rng, 1, 96)
        q = _log(rng, 8, 8000 // B) if long else rng.choice([1, 1, 3, 6])
        return _app("", B, (max(1, q // 3), q), (0, _log(rng, 1, 4000)), Hq, Hkv,
                    rng.choice([Hkv, 16]), layout, dtype,
                    rng.choice(["same", "e4m3", "i8", "mxfp4", "none"]),
                    rng.choice([32, 64, 128]), rng.choice(["halves", "interleaved"]), lengths)
    # new tokens x visible keys x heads, below the largest listed chunk's
    most = 2_000_000_000
    if op == "prompt":
        B = _log(rng, 1, 10)
        q = _log(rng, 16, min(6000, int(math.sqrt(most / (Hq * B)))))
        return _attn("", op, B, (1 if rng.random() < 0.5 else max(1, q // 3), q), (0, 0), Hq, Hkv,
                     layout, dtype, rng.choice([3, 3, 0]), 0, lengths)
    k = _log(rng, 1, 32) if op == "selected" else 0
    if long:
        B = _log(rng, 1, 6)
        q = _log(rng, 16, 2000 // B)
        ctx = _log(rng, 64, min(30000 // B, most // (B * q * Hq)))
        return _attn("", op, B, (max(1, q // 4), q), (ctx // 3, ctx), Hq, Hkv, layout, dtype,
                     rng.choice([3, 3, 0]), k, lengths)
    B = _log(rng, 1, 64)
    return _attn("", op, B, (1, rng.choice([1, 1, 2, 5])), (1, _log(rng, 100, 8000)), Hq, Hkv,
                 layout, dtype, 3, k, lengths)


def _lengths(case):
    """(new tokens, visible keys with the new ones) of each request."""
    rng = random.Random(case["lengths"])
    q = [_log(rng, case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    c = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    return q, [a + b for a, b in zip(q, c)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    q_lens, kv_lens = _lengths(case)
    B, T = len(q_lens), sum(q_lens)
    dt = TYPES[case["dtype"]]
    Hq, Hkv, layout = case["Hq"], case["Hkv"], case["layout"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=dt)

    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    s = {"case": case, "T": T, "q_max": max(q_lens), "kv_max": max(kv_lens),
         "cu": torch.tensor(cu, dtype=torch.int32, device=DEV),
         "kv": torch.tensor(kv_lens, dtype=torch.int32, device=DEV), "table": None}
    nb = [-(-n // P) for n in kv_lens]
    if layout != "TND":
        # the requests' pages lie scattered over a cache with some to spare;
        # the table's entries behind a request's last block name no page
        pages = sum(nb) + 3 + sum(nb) // 16
        perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
        table = torch.full((B, max(nb)), -1, dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(nb):
            table[b, :n] = perm[at:at + n]
            at += n
        s["table"] = table
        cache = lambda H, last: (pages, P, H, last) if layout == "BBND" else (pages, H, P, last)  # noqa: E731
    if case["op"] == "append":
        return _prepare_append(case, s, gen, normal, cache)
    # a fused projection's rows hold the queries (and a whole prompt's keys
    # and values) side by side
    if case["op"] == "prompt":
        qkv = normal(T, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        s["q"] = normal(T, Hq, D)
        s["k"], s["v"] = normal(*cache(Hkv, D)), normal(*cache(Hkv, D))
    if case["op"] == "selected":
        s["blocks"] = _select(case, s, gen, max(nb))
    return s


def _select(case, s, gen, nb):
    """[T, Hkv, k] ascending block numbers with a -1 tail, as the top-k of block
    scores gives them: the token's own block and the first one always, the rest
    by scores that neighbouring tokens share in part."""
    T, H, k = s["T"], case["Hkv"], case["k"]
    b, _, last = _rows(s, case["mode"])
    part = torch.randn((T + 63) // 64, H, nb, generator=gen, device=DEV)
    score = part[torch.arange(T, device=DEV) // 64]
    score = score + 0.5 * torch.randn(T, H, nb, generator=gen, device=DEV)
    blk = torch.arange(nb, device=DEV)
    own_blk = (last // P)[:, None, None]
    score = torch.where(blk == 0, 1e29, score)
    score = torch.where(blk == own_blk, 1e30, score)
    score = torch.where(blk > own_blk, -math.inf, score)
    top = score.topk(min(k, nb), dim=-1)
    idx = torch.where(top.values == -math.inf, 1 << 30, top.indices).sort(dim=-1).values
    idx = torch.where(idx == 1 << 30, -1, idx).to(torch.int32)
    out = torch.full((T, H, k), -1, dtype=torch.int32, device=DEV)
    out[..., :idx.shape[-1]] = idx
    return out


def _prepare_append(case, s, gen, normal, cache):
    T, Hq, Hkv, Hi, dt = s["T"], case["Hq"], case["Hkv"], case["Hi"], TYPES[case["dtype"]]
    rot, index = case["rot"], case["index"]
    # angles of every position, as a model keeps them
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    ang = torch.arange(s["kv_max"], dtype=torch.float64, device=DEV)[:, None] * inv
    s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    qkv = normal(T, Hq + 2 * Hkv, D)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device=DEV)
    s["k_cache"], s["v_cache"] = normal(*cache(Hkv, D)), normal(*cache(Hkv, D))
    if index == "none":
        return s
    iqk = normal(T, Hi + 1, D)
    s["iq"], s["ik"] = iqk[:, :Hi], iqk[:, Hi:]
    s["iq_scale"] = s["ik_scale"] = None
    if index == "mxfp4":
        s["iq_out"] = torch.zeros(T, Hi, D // 2, dtype=torch.uint8, device=DEV)
        s["iq_scale"] = torch.zeros(T, Hi, D // 32, dtype=torch.uint8, device=DEV)
        s["ik_cache"] = torch.zeros(cache(1, D // 2), dtype=torch.uint8, device=DEV)
        s["ik_scale"] = torch.zeros(cache(1, D // 32), dtype=torch.uint8, device=DEV)
        return s
    ct = {"same": dt, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}[index]
    s["iq_out"] = torch.empty(T, Hi, D, dtype=dt if index == "i8" else ct, device=DEV)
    s["ik_cache"] = torch.zeros(cache(1, D), dtype=ct, device=DEV)
    if index == "i8":
        pages = s["ik_cache"].shape[0]
        s["ik_scale"] = torch.zeros(pages, 1, P, dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        return _own_append(s) if op == "append" else _own_attention(s)
    if op == "append":
        return _plain_append(s)
    return _plain_selected(s) if op == "selected" else _plain_attention(s)


def _own_append(s):
    import block_max_qk_amd as m
    c = s["case"]
    items = [m.CacheItem(s["q"], s["q_out"], "ROWS", rotate=True),
             m.CacheItem(s["k"], s["k_cache"], c["layout"], rotate=True),
             m.CacheItem(s["v"], s["v_cache"], c["layout"])]
    if c["index"] != "none":
        items += [m.CacheItem(s["iq"], s["iq_out"], "ROWS", scale=s["iq_scale"], rotate=True),
                  m.CacheItem(s["ik"], s["ik_cache"], c["layout"], scale=s["ik_scale"],
                              rotate=True)]
    m.msa_cache_append(items, s["cos"], s["sin"], s["table"], s["cu"], s["kv"],
                       interleaved=c["pairs"] == "interleaved")
    return _append_outputs(s)


def _own_attention(s):
    import block_max_qk_amd as m
    c = s["case"]
    if c["op"] == "selected":
        out, lse = m.block_attention(s["q"], s["k"], s["v"], s["blocks"], s["table"], s["cu"],
                                     s["kv"], c["layout"], sparse_mode=c["mode"], return_lse=True)
    else:
        out, lse = m.attention(s["q"], s["k"], s["v"], s["table"], s["cu"], s["kv"], c["layout"],
                               sparse_mode=c["mode"], return_lse=True)
    return {"out": out, "lse": lse}


def _rows(s, mode=3):
    """(request, position in the sequence, last visible key) of every token."""
    t = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(s["cu"][1:].contiguous(), t, right=True)
    kv, cu = s["kv"].long(), s["cu"].long()
    pos = kv[b] - (cu[b + 1] - cu[b]) + t - cu[b]
    return b, pos, pos if mode == 3 else kv[b] - 1


# --- the append -------------------------------------------------------------


def _rotated(x, cos, sin, pairs, wide):
    """x [T, H, D] with its first elements rotated by the angles [T, rot / 2]."""
    x = x.to(wide)
    c, n = cos.to(wide)[:, None], sin.to(wide)[:, None]
    rot = 2 * c.shape[-1]
    if pairs == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * c - b * n, b * c + a * n], dim=-1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * n, b * c + a * n], dim=-1).flatten(-2)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _codes_i8(y):
    amax = y.abs().amax(dim=-1, keepdim=True)
    scale = (amax / 127).float()
    code = torch.round(y / torch.where(scale == 0, 1.0, scale).double()).clamp(-127, 127)
    return code.to(torch.int8), scale[..., 0]


def _codes_mxfp4(y):
    g = y.unflatten(-1, (D // 32, 32))
    amax = g.abs().amax(dim=-1)
    e = (torch.frexp(amax).exponent - 1 - 2 + 127).clamp(0, 254)
    e = torch.where(amax == 0, 0, e)
    a = (g * torch.exp2(127.0 - e.double())[..., None])
    m = a.abs()
    idx = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5)
           + (m >= 3.5) + (m > 5))
    nib = (idx + 8 * ((a < 0) & (idx > 0))).flatten(-2)
    return (nib[..., 0::2] | (nib[..., 1::2] << 4)).to(torch.uint8), e.to(torch.uint8)


def _e4m3(y):
    return y.float().clamp(-448, 448).to(torch.float8_e4m3fn)


def _put(cache, rows, layout, page, slot):
    """cache[page, slot] = rows (one per token), in the cache's layout."""
    bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[cache.element_size()]
    cache, rows = cache.view(bits), rows.contiguous().view(bits)
    if layout == "BBND":
        cache[page, slot] = rows
    else:
        cache[page, :, slot] = rows


def _plain_append(s):
    c = s["case"]
    b, pos, _ = _rows(s)
    cos, sin, pairs = s["cos"][pos], s["sin"][pos], c["pairs"]
    page = s["table"][b, pos // P].long()
    slot, lay, dt, f32, f64 = pos % P, c["layout"], TYPES[c["dtype"]], torch.float32, torch.float64
    s["q_out"].copy_(_rotated(s["q"], cos, sin, pairs, f32).to(dt))
    _put(s["k_cache"], _rotated(s["k"], cos, sin, pairs, f32).to(dt), lay, page, slot)
    _put(s["v_cache"], s["v"], lay, page, slot)
    if c["index"] == "same":
        s["iq_out"].copy_(_rotated(s["iq"], cos, sin, pairs, f32).to(dt))
        _put(s["ik_cache"], _rotated(s["ik"], cos, sin, pairs, f32).to(dt), lay, page, slot)
    elif c["index"] == "e4m3":
        s["iq_out"].copy_(_e4m3(_rotated(s["iq"], cos, sin, pairs, f64)))
        _put(s["ik_cache"], _e4m3(_rotated(s["ik"], cos, sin, pairs, f64)), lay, page, slot)
    elif c["index"] == "i8":
        s["iq_out"].copy_(_rotated(s["iq"], cos, sin, pairs, f32).to(dt))
        code, scale = _codes_i8(_rotated(s["ik"], cos, sin, pairs, f64))
        _put(s["ik_cache"], code, lay, page, slot)
        s["ik_scale"][page, :, slot] = scale
    elif c["index"] == "mxfp4":
        code, scale = _codes_mxfp4(_rotated(s["iq"], cos, sin, pairs, f64))
        s["iq_out"].copy_(code)
        s["iq_scale"].copy_(scale)
        code, scale = _codes_mxfp4(_rotated(s["ik"], cos, sin, pairs, f64))
        _put(s["ik_cache"], code, lay, page, slot)
        _put(s["ik_scale"], scale, lay, page, slot)
    return _append_outputs(s)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _values_mxfp4(code, scale):
    """The numbers that E2M1 pairs and their E8M0 scales stand for."""
    lut = torch.tensor(_E2M1 + [-x for x in _E2M1], device=DEV)
    v = torch.stack([lut[(code & 15).long()], lut[(code >> 4).long()]], dim=-1)
    v = v.flatten(-2).unflatten(-1, (D // 32, 32))
    return (v * torch.exp2(scale.float() - 127)[..., None]).flatten(-2)


def _append_outputs(s):
    out = {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    index = s["case"]["index"]
    if index in ("same", "e4m3"):
        out |= {"iq": s["iq_out"], "ik_cache": s["ik_cache"]}
    elif index == "i8":
        scale = s["ik_scale"] if s["case"]["layout"] == "BNBD" else s["ik_scale"].transpose(1, 2)
        out |= {"iq": s["iq_out"], "ik_cache": s["ik_cache"].float() * scale[..., None]}
    elif index == "mxfp4":
        out |= {"iq": _values_mxfp4(s["iq_out"], s["iq_scale"]),
                "ik_cache": _values_mxfp4(s["ik_cache"], s["ik_scale"])}
    return out


# --- the attention ----------------------------------------------------------


def _padded(s, x):
    """Keys or values of every request, [B, Hkv, keys, D] in 32 bits, padded to
    the longest request (the padding holds some row's values)."""
    c = s["case"]
    if c["layout"] == "TND":
        kv = s["kv"].long()
        first = kv.cumsum(0) - kv
        j = torch.arange(s["kv_max"], device=DEV)
        rows = (first[:, None] + j).clamp(max=x.shape[0] - 1)
        return x[rows].float().transpose(1, 2).contiguous()
    y = x[s["table"].clamp(min=0).long()]
    if c["layout"] == "BBND":
        return y.flatten(1, 2).float().transpose(1, 2).contiguous()
    return y.transpose(1, 2).flatten(2, 3).float().contiguous()


def _weights(score, visible):
    """(exp(score - max), its sum, log of the sum of exps) along the last axis."""
    score = torch.where(visible, score, -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(dim=-1, keepdim=True)
    return p, total, top + torch.log(total)


def _plain_attention(s):
    c = s["case"]
    Hq, Hkv = c["Hq"], c["Hkv"]
    g = Hq // Hkv
    b, pos, last = _rows(s, c["mode"])
    B, Q, i = c["B"], s["q_max"], torch.arange(s["T"], device=DEV) - s["cu"].long()[b]
    q = torch.zeros(B, Q, Hq, D, device=DEV)
    q[b, i] = s["q"].float()
    end = torch.full((B, Q), -1, device=DEV)
    end[b, i] = last
    q = q.view(B, Q, Hkv, g, D).transpose(1, 2).reshape(B, Hkv, Q * g, D)
    k, v = _padded(s, s["k"]), _padded(s, s["v"])
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) / math.sqrt(D)
    j = torch.arange(k.shape[2], device=DEV)
    visible = j <= end.repeat_interleave(g, dim=1)[:, None, :, None]
    p, total, lse = _weights(score, visible)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    out = out.view(B, Hkv, Q, g, D).transpose(1, 2).reshape(B, Q, Hq, D)[b, i]
    lse = lse.view(B, Hkv, Q, g).transpose(1, 2).reshape(B, Q, Hq)[b, i]
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _plain_selected(s):
    c = s["case"]
    T, Hq, Hkv, k = s["T"], c["Hq"], c["Hkv"], c["k"]
    b, pos, last = _rows(s, c["mode"])
    blocks = s["blocks"].long()                                     # [T, Hkv, k]
    page = s["table"][b[:, None, None], blocks.clamp(min=0)].clamp(min=0).long()
    h = torch.arange(Hkv, device=DEV)[:, None]
    if c["layout"] == "BBND":
        keys, vals = s["k"][page, :, h], s["v"][page, :, h]         # [T, Hkv, k, P, D]
    else:
        keys, vals = s["k"][page, h], s["v"][page, h]
    q = s["q"].float().view(T, Hkv, Hq // Hkv, D)
    keys = keys.flatten(2, 3).float().transpose(2, 3).contiguous()
    score = torch.matmul(q, keys) / math.sqrt(D)
    j = blocks[..., None] * P + torch.arange(P, device=DEV)
    visible = ((blocks >= 0)[..., None] & (j <= last[:, None, None, None])).flatten(2)
    p, total, lse = _weights(score, visible[:, :, None])
    out = torch.matmul(p, vals.flatten(2, 3).float()) / torch.where(total == 0, 1.0, total)
    return {"out": out.view(T, Hq, D).to(s["q"].dtype), "lse": lse.view(T, Hq)}


# ---------------------------------------------------------------------------
# work and the definition in 64 bits
# ---------------------------------------------------------------------------


def work(case):
    q_lens, kv_lens = _lengths(case)
    T, Hq, Hkv = sum(q_lens), case["Hq"], case["Hkv"]
    if case["op"] == "append":
        rows = Hq + 2 * Hkv
        moved = T * rows * D * 4 + T * case["rot"] * 4
        flops = T * (Hq + Hkv) * case["rot"] * 3
        if case["index"] != "none":
            size = {"same": (2, 2), "e4m3": (1, 1), "i8": (2, 1 + 4 / D),
                    "mxfp4": (17 / 32, 17 / 32)}[case["index"]]
            moved += T * D * (case["Hi"] * (2 + size[0]) + 2 + size[1])
            flops += T * (case["Hi"] + 1) * case["rot"] * 3
        return {"bytes": moved, "flops": flops}
    keys = pairs = 0
    for n, kv in zip(q_lens, kv_lens):
        ends = [kv - n + i if case["mode"] == 3 else kv - 1 for i in range(n)]
        if case["op"] == "selected":
            read = [(min(case["k"], e // P + 1) - 1) * P + e % P + 1 for e in ends]
            keys += min(kv, sum(read))
            pairs += sum(read)
        else:
            keys += kv
            pairs += sum(e + 1 for e in ends)
    moved = 4 * keys * Hkv * D + 4 * T * Hq * D + 4 * T * Hq + 4 * T * Hkv * case["k"]
    return {"bytes": moved, "flops": 4 * pairs * Hq * D}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


def _exact_append(s):
    c = s["case"]
    T, rot, kv = s["T"], c["rot"], s["kv"].tolist()
    cu = s["cu"].tolist()
    where = [(b, kv[b] - (cu[b + 1] - cu[b]) + i) for b in range(c["B"])
             for i in range(cu[b + 1] - cu[b])]
    at = torch.tensor([w[1] for w in where], device=DEV)
    page = s["table"][torch.tensor([w[0] for w in where], device=DEV), at // P].long()
    # rotation of pair (a, b) as a complex product
    turn = torch.complex(s["cos"].double(), s["sin"].double())[at][:, None]

    def turned(x):
        x = x.double().clone()
        if c["pairs"] == "halves":
            z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous())
            z = z * turn
            x[..., :rot // 2], x[..., rot // 2:rot] = z.real, z.imag
        else:
            z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * turn
            x[..., 0:rot:2], x[..., 1:rot:2] = z.real, z.imag
        return x

    def stored(cache, rows):
        full = cache.double()
        view = full if c["layout"] == "BBND" else full.transpose(1, 2)
        view[page, at % P] = rows
        return full

    out = {"q": turned(s["q"]), "k_cache": stored(s["k_cache"], turned(s["k"])),
           "v_cache": stored(s["v_cache"], s["v"].double())}
    if c["index"] in ("same", "i8"):
        out["iq"] = turned(s["iq"])
    if c["index"] == "same":
        out["ik_cache"] = stored(s["ik_cache"], turned(s["ik"]))
    elif c["index"] == "e4m3":
        out["iq"] = turned(s["iq"])
        out["ik_cache"] = stored(s["ik_cache"], turned(s["ik"]))
    elif c["index"] == "i8":
        x = turned(s["ik"])
        step = (x.abs().amax(-1, keepdim=True) / 127).float().double()
        out["ik_cache"] = stored(torch.zeros_like(s["ik_cache"], dtype=torch.float64),
                                 torch.round(x / step) * step)
    elif c["index"] == "mxfp4":
        grid = torch.tensor(_E2M1, dtype=torch.float64, device=DEV)
        # ties go to the code with an even last bit
        tie = 1e-9 * (torch.arange(8, device=DEV) % 2)

        def nearest(x):
            y = x.reshape(-1, 32)
            step = 2.0 ** (torch.floor(torch.log2(y.abs().amax(-1, keepdim=True))) - 2)
            near = ((y / step).abs()[..., None] - grid).abs() + tie
            return (torch.sign(y) * grid[near.argmin(-1)] * step).reshape(x.shape)

        out["iq"] = nearest(turned(s["iq"]))
        shape = s["ik_cache"].shape[:-1] + (D,)
        out["ik_cache"] = stored(torch.zeros(shape, dtype=torch.float64, device=DEV),
                                 nearest(turned(s["ik"])))
    return out


def _exact_attention(s):
    c = s["case"]
    Hq, Hkv, T = c["Hq"], c["Hkv"], s["T"]
    g = Hq // Hkv
    if work(c)["flops"] > 6e12:
        return None
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    cu, kv, first = s["cu"].tolist(), s["kv"].tolist(), 0
    for b in range(c["B"]):
        n, L = cu[b + 1] - cu[b], kv[b]
        nb = -(-L // P)
        i = torch.arange(n, device=DEV)
        end = L - n + i if c["mode"] == 3 else torch.full_like(i, L - 1)
        seen = torch.arange(L, device=DEV)[None] <= end[:, None]
        for h in range(Hkv):
            if c["layout"] == "TND":
                key, val = s["k"][first:first + L, h], s["v"][first:first + L, h]
            elif c["layout"] == "BBND":
                pages = s["table"][b, :nb].long()
                key, val = s["k"][pages, :, h], s["v"][pages, :, h]
            else:
                pages = s["table"][b, :nb].long()
                key, val = s["k"][pages, h], s["v"][pages, h]
            key, val = (x.reshape(-1, D)[:L].double() for x in (key, val))
            mine = seen
            if c["op"] == "selected":
                chosen = torch.zeros(n, nb + 1, dtype=torch.bool, device=DEV)
                names = s["blocks"][cu[b]:cu[b + 1], h].long()
                chosen.scatter_(1, torch.where(names < 0, nb, names), True)
                mine = seen & chosen[:, :nb].repeat_interleave(P, dim=1)[:, :L]
            for r in range(h * g, (h + 1) * g):
                x = s["q"][cu[b]:cu[b + 1], r].double() @ key.T.contiguous() * D ** -0.5
                x = x.masked_fill(~mine, -math.inf)
                z = torch.logsumexp(x, dim=-1)
                lse[cu[b]:cu[b + 1], r] = z
                w = torch.where(mine, (x - z[:, None]).exp(), 0.0)
                out[cu[b]:cu[b + 1], r] = w @ val
        first += L
    return {"out": out, "lse": lse}
