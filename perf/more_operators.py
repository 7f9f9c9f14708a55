"""More serving operators around the index branch, as cases to measure.

Three operators of one step of a server whose prompts hold images or documents
and whose models cap their scores or weigh them by distance:

- the step's tables: from the requests' lengths the prefix sums, block tables,
  positions and slots that every other operator here takes, with pages from a
  free list for the blocks that the new tokens begin;
- the cache append with several position axes (time, height, width), where each
  rotated pair turns by the position of its own axis;
- attention over a paged or packed cache with scores capped by a tanh, with a
  bias that falls with the distance, and with a range of visible keys per token
  (documents, images that see themselves whole, prefixes).

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
# op        tables | append | attention
# B, q_lo, q_hi, ctx_lo, ctx_hi
#           requests; new tokens and earlier tokens of each are drawn from
#           these ranges (over their logarithm, and evenly) by a generator of
#           the case's own ("lengths"), so the sizes do not depend on the seed
# MB, R, pad, spare
#           tables: width of the block tables, rows of the server's pool, rows
#           behind the last token, free pages beyond what the step needs
# Hq, Hkv   query and key/value heads; layout of the cache; mode 3 is causal
# index, Hi the append's index branch and its query heads
# rot, pairs, axes, mix
#           rotated elements, how they pair up, position axes, and whether an
#           axis has a run of pairs ("runs") or every axes-th one ("turns")
# cap, bias, mask
#           largest score (0: none), a slope per head or not, and what narrows
#           the keys that a token sees: none | documents | images | prefix


def _tab(name, B, q, ctx, MB, R, pad=0, spare=64, lengths=1):
    return {"name": name, "op": "tables", "B": B, "q_lo": q[0], "q_hi": q[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "MB": MB, "R": R, "pad": pad, "spare": spare, "lengths": lengths}


def _app(name, B, q, ctx, Hq, Hkv, Hi, layout, dtype, index, rot, pairs, axes, mix, lengths=1):
    return {"name": name, "op": "append", "B": B, "q_lo": q[0], "q_hi": q[1], "ctx_lo": ctx[0],
            "ctx_hi": ctx[1], "Hq": Hq, "Hkv": Hkv, "Hi": Hi, "layout": layout, "dtype": dtype,
            "index": index, "rot": rot, "pairs": pairs, "axes": axes, "mix": mix,
            "lengths": lengths}


def _attn(name, B, q, ctx, Hq, Hkv, layout, dtype, cap=0.0, bias=False, mask="none", mode=3,
          lengths=1):
    return {"name": name, "op": "attention", "B": B, "q_lo": q[0], "q_hi": q[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "Hq": Hq, "Hkv": Hkv, "layout": layout,
            "dtype": dtype, "cap": cap, "bias": bias, "mask": mask, "mode": mode,
            "lengths": lengths}


def listed():
    return [
        # a decode step's tables: 64 requests, one new token each
        _tab("tables_decode", 64, (1, 1), (1, 8191), 256, 256),
        # a scheduler's mixed step: decode tokens beside chunks, rows of a
        # larger pool, a batch padded for a captured graph
        _tab("tables_mixed", 300, (1, 200), (0, 32000), 1024, 1024, 512),
        # a wide decode step over long tables
        _tab("tables_wide", 4096, (1, 2), (1, 32767), 1024, 5000),
        # one decode step of 64 requests, three axes by runs of pairs
        _app("axes_decode_bf16", 64, (1, 1), (1, 4095), 32, 4, 4, "BBND", "bf16", "same", 128,
             "halves", 3, "runs"),
        # four prompts with images, axes by turns, fp8 index rows
        _app("axes_prefill_e4m3", 4, (1000, 8192), (0, 4096), 64, 8, 8, "BBND", "bf16", "e4m3",
             64, "halves", 3, "turns"),
        # the smallest capped chunk: 32 new tokens in two blocks
        _attn("capped_tiny_f16", 1, (32, 32), (224, 224), 8, 1, "BBND", "f16", 30.0),
        # a decode batch of a model that caps its scores
        _attn("capped_decode_bf16", 64, (1, 1), (1, 8191), 64, 8, "BBND", "bf16", 50.0),
        # a chunk of a long prompt of such a model
        _attn("capped_chunk_bf16", 1, (2048, 2048), (30720, 30720), 32, 4, "BBND", "bf16", 50.0),
        # a decode batch with a slope per head over long contexts
        _attn("biased_decode_f16", 24, (1, 1), (1, 30000), 32, 4, "BNBD", "f16", 0.0, True),
        # whole prompts with a slope per head, packed
        _attn("biased_prompt_bf16", 5, (150, 8192), (0, 0), 32, 4, "TND", "bf16", 0.0, True),
        # two long prompts of many documents that do not see one another
        _attn("documents_bf16", 2, (6000, 8192), (0, 2000), 32, 4, "BBND", "bf16",
              mask="documents"),
        # a mixed batch of prompts with images, capped
        _attn("images_f16", 9, (1, 700), (1, 6000), 32, 4, "BNBD", "f16", 30.0, False, "images",
              0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 1)),
                                                          math.log(max(hi, 1))))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attention", "attention", "attention"])
    lengths = rng.randrange(1 << 20)
    if op == "tables":
        B = _log(rng, 1, 3000)
        q = _log(rng, 1, max(1, min(8000, 30000 // B)))
        MB = _log(rng, 4, 1000)
        ctx = _log(rng, 1, MB * P)
        return _tab("", B, (rng.choice([0, 1, q]), q), (rng.choice([0, ctx // 2]), ctx), MB,
                    B + _log(rng, 1, 500), rng.choice([0, _log(rng, 1, 1000)]),
                    rng.choice([100, 1, 0, -3]), lengths)
    dtype = rng.choice(["bf16", "f16"])
    Hq, Hkv = rng.choice([(8, 1), (16, 1), (32, 4), (64, 8), (12, 4), (10, 2), (8, 8)])
    long = rng.random() < 0.5
    if op == "append":
        B = _log(rng, 1, 8) if long else _log(rng, 1, 96)
        q = _log(rng, 8, 8000 // B) if long else rng.choice([1, 1, 3, 6])
        return _app("", B, (max(1, q // 3), q), (0, _log(rng, 1, 4000)), Hq, Hkv,
                    rng.choice([Hkv, 16]), rng.choice(["BBND", "BNBD"]), dtype,
                    rng.choice(["same", "e4m3", "none"]), rng.choice([32, 64, 128]),
                    rng.choice(["halves", "interleaved"]), rng.choice([1, 2, 3, 3, 4]),
                    rng.choice(["runs", "turns"]), lengths)
    cap = rng.choice([0.0, 20.0, 30.0, 50.0])
    bias = rng.random() < 0.4
    mask = rng.choice(["none", "documents", "images", "prefix"])
    mode = 3 if mask in ("none", "documents") else 0
    layout = rng.choice(["TND", "BBND", "BBND", "BNBD", "BNBD"])
    # new tokens x keys x heads, below the largest listed chunk's
    most = 1_900_000_000
    if layout == "TND":
        B = _log(rng, 1, 10)
        q = _log(rng, 16, min(6000, int(math.sqrt(most / (Hq * B)))))
        return _attn("", B, (1 if rng.random() < 0.5 else max(1, q // 3), q), (0, 0), Hq, Hkv,
                     layout, dtype, cap, bias, mask, mode, lengths)
    if long:
        B = _log(rng, 1, 6)
        q = _log(rng, 16, 2000 // B)
        ctx = _log(rng, 64, max(64, min(30000 // B, most // (B * q * Hq) - q)))
        return _attn("", B, (max(1, q // 4), q), (ctx // 3, ctx), Hq, Hkv, layout, dtype, cap,
                     bias, mask, mode, lengths)
    B = _log(rng, 1, 64)
    return _attn("", B, (1, rng.choice([1, 1, 2, 5])), (1, _log(rng, 100, 8000)), Hq, Hkv, layout,
                 dtype, cap, bias, mask, mode, lengths)


def _lengths(case):
    """(new tokens, earlier tokens) of each request."""
    rng = random.Random(case["lengths"])
    q = [_log(rng, case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    c = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    if case["op"] == "tables" and case["q_lo"] == 0:   # some requests bring nothing
        q = [0 if rng.random() < 0.2 else n for n in q]
    return q, c


def _ranges(case):
    """(first visible key, end of them) of every new token."""
    rng = random.Random(case["lengths"] + 1)
    out = []
    for n, c in zip(*_lengths(case)):
        kv = n + c
        if case["mask"] == "documents":     # documents of 40 to 2000 tokens
            at = 0
            while at < kv:
                end = min(kv, at + _log(rng, 40, 2000))
                out += [(at, end)] * max(0, end - max(at, c))
                at = end
        elif case["mask"] == "images":      # text of 5 to 400 tokens, images of 64 to 1024
            at, image = 0, False
            while at < kv:
                end = min(kv, at + (_log(rng, 64, 1024) if image else _log(rng, 5, 400)))
                out += [(0, end if image else p + 1) for p in range(max(at, c), end)]
                at, image = end, not image
        elif case["mask"] == "prefix":
            prefix = rng.randint(0, kv)
            out += [(0, max(p + 1, prefix)) for p in range(c, kv)]
        else:
            out += [(0, p + 1) for p in range(c, kv)]
    return out


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"tables": _prepare_tables, "append": _prepare_append,
            "attention": _prepare_attention}[case["op"]](case, gen)


def _prepare_tables(case, gen):
    q, c = _lengths(case)
    B, MB, R = case["B"], case["MB"], case["R"]
    held = [min(MB, -(-n // P)) for n in c]
    need = sum(min(MB, -(-(n + m) // P)) - h for n, m, h in zip(c, q, held))
    free = max(0, need + case["spare"])
    s = {"case": case, "T": sum(q) + case["pad"], "new": _i32(q), "ctx": _i32(c)}
    # the requests' rows lie scattered over the pool, their pages over the cache
    s["rows"] = torch.randperm(R, generator=gen, device=DEV)[:B].to(torch.int32)
    pages = torch.randperm(sum(held) + free, generator=gen, device=DEV).to(torch.int32)
    s["pool"] = torch.full((R, MB), -1, dtype=torch.int32, device=DEV)
    live = torch.arange(MB, device=DEV) < _i32(held)[:, None]
    mine = torch.full((B, MB), -1, dtype=torch.int32, device=DEV)
    mine[live] = pages[:sum(held)]
    s["pool"][s["rows"].long()] = mine
    # a free list with room for every page
    s["free"] = torch.full((len(pages),), -1, dtype=torch.int32, device=DEV)
    s["free"][:free] = pages[sum(held):]
    s["count"] = _i32([free, 0])
    # what the step is written to, which a server keeps
    size = {"cu_seqlens_q": (B + 1,), "kv_len": (B,), "start_loc": (B,), "block_table": (B, MB),
            "positions": (s["T"],), "slots": (s["T"],), "cu_pages": (B + 1,)}
    s["out"] = {n: torch.empty(shape, dtype=torch.int64 if n == "slots" else torch.int32,
                               device=DEV) for n, shape in size.items()}
    s["left"] = torch.empty_like(s["count"])
    return s


def _paged(case, s, gen):
    """The block tables of scattered pages, and a cache's shape."""
    nb = [-(-n // P) for n in s["kv_list"]]
    pages = sum(nb) + 3 + sum(nb) // 16
    perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    s["table"] = torch.full((case["B"], max(nb)), -1, dtype=torch.int32, device=DEV)
    s["table"][torch.arange(max(nb), device=DEV) < _i32(nb)[:, None]] = perm[:sum(nb)]
    if case["layout"] == "BBND":
        return lambda H: (pages, P, H, D)
    return lambda H: (pages, H, P, D)


def _lens(case):
    q, c = _lengths(case)
    kv = [a + b for a, b in zip(q, c)]
    cu = [0]
    for n in q:
        cu.append(cu[-1] + n)
    return {"case": case, "T": cu[-1], "q_max": max(q), "kv_max": max(kv), "kv_list": kv,
            "cu_list": cu, "cu": _i32(cu), "kv": _i32(kv), "table": None}


def _pair_axes(case):
    """The axis of each rotated pair: runs of pairs (the first axis has the
    longest), or every axes-th pair."""
    half, axes = case["rot"] // 2, case["axes"]
    if case["mix"] == "turns":
        return [r % axes for r in range(half)]
    run = half // axes
    return [max(0, (r - (half - run * axes)) // run) for r in range(half)]


def _prepare_append(case, gen):
    s = _lens(case)
    T, Hq, Hkv, Hi, dt = s["T"], case["Hq"], case["Hkv"], case["Hi"], TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=dt)

    cache = _paged(case, s, gen)
    inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEV)
                      / case["rot"])
    ang = torch.arange(s["kv_max"], dtype=torch.float64, device=DEV)[:, None] * inv
    s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    # the first axis follows the sequence, the others a frame's rows and columns
    _, pos = _places(s)
    axes = [pos]
    for a in range(1, case["axes"]):
        side = torch.randint(0, 64, (T,), generator=gen, device=DEV)
        axes.append(torch.minimum(pos // (2 * a) + side, pos))
    s["axis_pos"] = torch.stack(axes).to(torch.int32)
    s["pair_axes"] = _pair_axes(case)
    qkv = normal(T, Hq + 2 * Hkv, D)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device=DEV)
    s["k_cache"], s["v_cache"] = normal(*cache(Hkv)), normal(*cache(Hkv))
    if case["index"] != "none":
        ct = dt if case["index"] == "same" else torch.float8_e4m3fn
        iqk = normal(T, Hi + 1, D)
        s["iq"], s["ik"] = iqk[:, :Hi], iqk[:, Hi:]
        s["iq_out"] = torch.empty(T, Hi, D, dtype=ct, device=DEV)
        s["ik_cache"] = torch.zeros(cache(1), dtype=ct, device=DEV)
    return s


def _prepare_attention(case, gen):
    s = _lens(case)
    T, Hq, Hkv, dt = s["T"], case["Hq"], case["Hkv"], TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    # heads are sharp to different degrees: scores of 0.4 to 8 in the mean square
    sharp = torch.exp(0.5 + 0.7 * normal(Hq)).clamp(0.4, 8.0)[:, None]
    if case["layout"] == "TND":
        qkv = normal(T, Hq + 2 * Hkv, D)
        qkv[:, :Hq] *= sharp
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        cache = _paged(case, s, gen)
        s["q"] = (normal(T, Hq, D) * sharp).to(dt)
        s["k"], s["v"] = normal(*cache(Hkv)).to(dt), normal(*cache(Hkv)).to(dt)
    s["slopes"] = s["visible"] = None
    if case["bias"]:
        s["slopes"] = torch.tensor([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)], device=DEV)
    if case["mask"] != "none":
        s["visible"] = _i32(_ranges(case))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if op == "tables":
        return _own_tables(s) if own else _plain_tables(s)
    if op == "append":
        return _own_append(s) if own else _plain_append(s)
    return _own_attention(s) if own else _plain_attention(s)


def _own_tables(s):
    import block_max_qk_amd as m
    m.msa_step_tables(s["new"], s["ctx"], s["pool"], s["free"], s["count"],
                      m.StepTables(**s["out"]), rows=s["rows"], free_out=s["left"])
    return {**s["out"], "free": s["left"], "pool": s["pool"]}


def _own_append(s):
    import block_max_qk_amd as m
    c = s["case"]
    items = [m.CacheItem(s["q"], s["q_out"], "ROWS", rotate=True),
             m.CacheItem(s["k"], s["k_cache"], c["layout"], rotate=True),
             m.CacheItem(s["v"], s["v_cache"], c["layout"])]
    if c["index"] != "none":
        items += [m.CacheItem(s["iq"], s["iq_out"], "ROWS", rotate=True),
                  m.CacheItem(s["ik"], s["ik_cache"], c["layout"], rotate=True)]
    m.msa_cache_append(items, s["cos"], s["sin"], s["table"], s["cu"], s["kv"],
                       interleaved=c["pairs"] == "interleaved", axis_positions=s["axis_pos"],
                       pair_axes=s["pair_axes"])
    return _append_outputs(s)


def _own_attention(s):
    import block_max_qk_amd as m
    c = s["case"]
    out, lse = m.attention(s["q"], s["k"], s["v"], s["table"], s["cu"], s["kv"], c["layout"],
                           sparse_mode=c["mode"], softcap=c["cap"], slopes=s["slopes"],
                           visible=s["visible"], return_lse=True)
    return {"out": out, "lse": lse}


# --- the tables -------------------------------------------------------------


def _plain_tables(s):
    c = s["case"]
    B, MB, T, i32 = c["B"], c["MB"], s["T"], torch.int32
    new, ctx, rows = s["new"].long(), s["ctx"].long(), s["rows"].long()
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    kv = ctx + new
    cu = torch.cat([zero, new.cumsum(0)])
    old, now = ((ctx + P - 1) // P).clamp(max=MB), ((kv + P - 1) // P).clamp(max=MB)
    count = s["count"][0].long()
    wanted = torch.cat([zero, (now - old).cumsum(0)])
    cu_pages = torch.minimum(wanted, count)
    # blocks that begin in this step take pages from the list's end
    blk = torch.arange(MB, device=DEV)
    nth = wanted[:-1, None] + blk - old[:, None]
    fresh = (blk >= old[:, None]) & (blk < now[:, None])
    page = s["free"][(count - 1 - nth).clamp(0, max(s["free"].numel() - 1, 0))]
    page = torch.where(nth < count, page, -1)
    mine = torch.where(fresh, page, s["pool"][rows])
    s["pool"][rows] = mine
    table = torch.where(blk < now[:, None], mine, -1).to(i32)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    held = b < B
    b = b.clamp(max=B - 1)
    pos = torch.where(held, ctx[b] + t - cu[b], 0)
    at = table[b, (pos // P).clamp(max=MB - 1)].long()
    slot = torch.where(held & (at >= 0) & (pos < MB * P), at * P + pos % P, -1)
    left = torch.stack([count - cu_pages[-1], wanted[-1] - cu_pages[-1]])
    return {"cu_seqlens_q": cu.to(i32), "kv_len": kv.to(i32), "start_loc": (ctx // P).to(i32),
            "block_table": table, "positions": pos.to(i32), "slots": slot,
            "cu_pages": cu_pages.to(i32), "free": left.to(i32), "pool": s["pool"]}


# --- the append -------------------------------------------------------------


def _places(s):
    """(request, position) of every token."""
    t = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(s["cu"][1:].contiguous(), t, right=True)
    kv, cu = s["kv"].long(), s["cu"].long()
    return b, kv[b] - (cu[b + 1] - cu[b]) + t - cu[b]


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


def _put(cache, rows, layout, page, slot):
    """cache[page, slot] = rows (one per token), in the cache's layout."""
    bits = {1: torch.uint8, 2: torch.int16}[cache.element_size()]
    cache, rows = cache.view(bits), rows.contiguous().view(bits)
    if layout == "BBND":
        cache[page, slot] = rows
    else:
        cache[page, :, slot] = rows


def _plain_append(s):
    c = s["case"]
    b, pos = _places(s)
    axis = torch.tensor(s["pair_axes"], device=DEV)
    at = s["axis_pos"].long()[axis].T                          # [T, rot / 2]
    pair = torch.arange(c["rot"] // 2, device=DEV)
    cos, sin, pairs = s["cos"][at, pair], s["sin"][at, pair], c["pairs"]
    page = s["table"][b, pos // P].long()
    slot, lay, dt, f32, f64 = pos % P, c["layout"], TYPES[c["dtype"]], torch.float32, torch.float64
    s["q_out"].copy_(_rotated(s["q"], cos, sin, pairs, f32).to(dt))
    _put(s["k_cache"], _rotated(s["k"], cos, sin, pairs, f32).to(dt), lay, page, slot)
    _put(s["v_cache"], s["v"], lay, page, slot)
    if c["index"] == "same":
        s["iq_out"].copy_(_rotated(s["iq"], cos, sin, pairs, f32).to(dt))
        _put(s["ik_cache"], _rotated(s["ik"], cos, sin, pairs, f32).to(dt), lay, page, slot)
    elif c["index"] == "e4m3":
        def e4m3(y):
            return y.float().clamp(-448, 448).to(torch.float8_e4m3fn)
        s["iq_out"].copy_(e4m3(_rotated(s["iq"], cos, sin, pairs, f64)))
        _put(s["ik_cache"], e4m3(_rotated(s["ik"], cos, sin, pairs, f64)), lay, page, slot)
    return _append_outputs(s)


def _append_outputs(s):
    out = {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["case"]["index"] != "none":
        out |= {"iq": s["iq_out"], "ik_cache": s["ik_cache"]}
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


def _plain_attention(s):
    c = s["case"]
    Hq, Hkv, B, Q = c["Hq"], c["Hkv"], c["B"], s["q_max"]
    g = Hq // Hkv
    b, pos = _places(s)
    i = torch.arange(s["T"], device=DEV) - s["cu"].long()[b]
    end = s["kv"].long()[b] if c["mode"] == 0 else pos + 1
    first = torch.zeros_like(pos)
    if s["visible"] is not None:
        first = s["visible"][:, 0].long()
        end = torch.minimum(end, s["visible"][:, 1].long())

    def rows(x, fill):                   # a figure of each token, for [B, 1, Q g, 1]
        y = torch.full((B, Q), fill, device=DEV)
        y[b, i] = x
        return y.repeat_interleave(g, dim=1)[:, None, :, None]

    q = torch.zeros(B, Q, Hq, D, device=DEV)
    q[b, i] = s["q"].float()
    q = q.view(B, Q, Hkv, g, D).transpose(1, 2).reshape(B, Hkv, Q * g, D)
    k, v = _padded(s, s["k"]), _padded(s, s["v"])
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) / math.sqrt(D)
    if c["cap"]:
        score = c["cap"] * torch.tanh(score / c["cap"])
    j = torch.arange(k.shape[2], device=DEV)
    if c["bias"]:
        slope = s["slopes"].view(Hkv, 1, g).expand(Hkv, Q, g).reshape(1, Hkv, Q * g, 1)
        score = score - slope * (rows(pos, 0) - j).abs()
    seen = (j >= rows(first, 0)) & (j < rows(end, 0))
    score = torch.where(seen, score, -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(dim=-1, keepdim=True)
    lse = top + torch.log(total)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    out = out.view(B, Hkv, Q, g, D).transpose(1, 2).reshape(B, Q, Hq, D)[b, i]
    lse = lse.view(B, Hkv, Q, g).transpose(1, 2).reshape(B, Q, Hq)[b, i]
    return {"out": out.to(s["q"].dtype), "lse": lse}


# ---------------------------------------------------------------------------
# work and the definition in 64 bits
# ---------------------------------------------------------------------------


def work(case):
    q, c = _lengths(case)
    T = sum(q)
    if case["op"] == "tables":
        now = [min(case["MB"], -(-(n + m) // P)) for n, m in zip(c, q)]
        fresh = sum(now) - sum(min(case["MB"], -(-n // P)) for n in c)
        moved = (case["B"] * (12 + 16 + 4 * case["MB"]) + 4 * sum(now) + 4 * fresh
                 + 12 * (T + case["pad"]))
        return {"bytes": moved, "flops": 0}
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "append":
        moved = T * (Hq + 2 * Hkv) * D * 4 + T * case["rot"] * 4 + 4 * T * case["axes"]
        flops = T * (Hq + Hkv) * case["rot"] * 3
        if case["index"] != "none":
            size = 2 if case["index"] == "same" else 1
            moved += T * D * (case["Hi"] + 1) * (2 + size)
            flops += T * (case["Hi"] + 1) * case["rot"] * 3
        return {"bytes": moved, "flops": flops}
    at = keys = pairs = 0
    ranges = _ranges(case)
    for n, m in zip(q, c):
        mine = ranges[at:at + n]
        at += n
        if case["mode"] == 3:
            mine = [(a, min(e, m + i + 1)) for i, (a, e) in enumerate(mine)]
        pairs += sum(e - a for a, e in mine)
        # keys that some token sees: the union of the ranges, which come in order
        last = 0
        for a, e in mine:
            keys += max(0, e - max(a, last))
            last = max(last, e)
    moved = (4 * keys * Hkv * D + 4 * T * Hq * D + 4 * T * Hq
             + (8 * T if case["mask"] != "none" else 0))
    return {"bytes": moved, "flops": 4 * pairs * Hq * D}


def exact(case, seed):
    if case["op"] == "tables":
        return None                      # whole numbers only
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)


def _exact_append(s):
    c = s["case"]
    rot, cu, kv = c["rot"], s["cu_list"], s["kv_list"]
    where = [(b, kv[b] - (cu[b + 1] - cu[b]) + i) for b in range(c["B"])
             for i in range(cu[b + 1] - cu[b])]
    at = torch.tensor([w[1] for w in where], device=DEV)
    page = s["table"][torch.tensor([w[0] for w in where], device=DEV), at // P].long()
    # rotation of pair (a, b) as a complex product, axis by axis
    angle = torch.complex(s["cos"].double(), s["sin"].double())
    turn = torch.empty(s["T"], rot // 2, dtype=torch.complex128, device=DEV)
    for r, a in enumerate(s["pair_axes"]):
        turn[:, r] = angle[s["axis_pos"][a].long(), r]
    turn = turn[:, None]

    def turned(x):
        x = x.double().clone()
        a, b = ((slice(0, rot // 2), slice(rot // 2, rot)) if c["pairs"] == "halves"
                else (slice(0, rot, 2), slice(1, rot, 2)))
        z = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * turn
        x[..., a], x[..., b] = z.real, z.imag
        return x

    def stored(cache, rows):
        full = cache.double()
        view = full if c["layout"] == "BBND" else full.transpose(1, 2)
        view[page, at % P] = rows
        return full

    out = {"q": turned(s["q"]), "k_cache": stored(s["k_cache"], turned(s["k"])),
           "v_cache": stored(s["v_cache"], s["v"].double())}
    if c["index"] != "none":
        out |= {"iq": turned(s["iq"]), "ik_cache": stored(s["ik_cache"], turned(s["ik"]))}
    return out


def _exact_attention(s):
    c = s["case"]
    Hq, Hkv, T = c["Hq"], c["Hkv"], s["T"]
    g = Hq // Hkv
    if 4 * sum((e - b) * n for b, e, n in zip(s["cu_list"], s["cu_list"][1:], s["kv_list"])) * (
            Hq * D) > 6e12:
        return None
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=DEV)
    cu, kv, start = s["cu_list"], s["kv_list"], 0
    for b in range(c["B"]):
        lo, hi, L = cu[b], cu[b + 1], kv[b]
        pos = L - (hi - lo) + torch.arange(hi - lo, device=DEV)[:, None]
        key_at = torch.arange(L, device=DEV)[None]
        hidden = key_at > pos if c["mode"] == 3 else torch.zeros_like(key_at > pos)
        if s["visible"] is not None:
            span = s["visible"][lo:hi]
            hidden = hidden | (key_at < span[:, :1]) | (key_at >= span[:, 1:])
        away = (pos - key_at).abs().double()
        pages = None if c["layout"] == "TND" else s["table"][b, :-(-L // P)].long()
        for h in range(Hkv):
            if pages is None:
                key, val = s["k"][start:start + L, h], s["v"][start:start + L, h]
            elif c["layout"] == "BBND":
                key, val = s["k"][pages, :, h], s["v"][pages, :, h]
            else:
                key, val = s["k"][pages, h], s["v"][pages, h]
            key, val = (x.reshape(-1, D)[:L].double() for x in (key, val))
            for r in range(h * g, (h + 1) * g):
                x = s["q"][lo:hi, r].double() @ key.T.contiguous() * D ** -0.5
                if c["cap"]:
                    x = torch.tanh(x / c["cap"]) * c["cap"]
                if c["bias"]:
                    x = x - float(s["slopes"][r]) * away
                x = x.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, dim=-1)
                lse[lo:hi, r] = z
                w = torch.where(hidden, 0.0, (x - z[:, None]).exp())
                out[lo:hi, r] = w @ val
        start += L
    return {"out": out, "lse": lse}
