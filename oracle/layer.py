"""CPU oracle of the operators around the index branch: the cache append and
the attention, dense or over selected blocks.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Everything is taken
in binary64 from the operators' definitions, one request and one head at a
time; no code is shared with the HIP library or its binding.
"""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import torch

P = 128
D = 128


def positions(cu, kv_len, T: int):
    """(t, request, position) of every token that a request holds."""
    cu, kv = [int(x) for x in cu], [int(x) for x in kv_len]
    for b in range(len(kv)):
        for t in range(cu[b], min(cu[b + 1], T)):
            yield t, b, kv[b] - (cu[b + 1] - cu[b]) + t - cu[b]


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------


class Attention(NamedTuple):
    out: torch.Tensor      # [T, Hq, D] float64
    lse: torch.Tensor      # [T, Hq] float64
    spread: torch.Tensor   # [T, Hq, D]: sum of |weight * value|, for error bounds
    size: torch.Tensor     # [T, Hq]: largest scale * sum |q k| of a visible key
    keys: torch.Tensor     # [T, Hq]: visible keys
    top: torch.Tensor      # [T, Hq]: largest |value| of a visible key


def request_rows(x, layout, block_table, b, length, first):
    """(rows [n, H, D], present [n]) of a request's keys or values; rows on
    pages that the table does not name, or behind the tensor, are not present."""
    if layout == "TND":
        n = max(0, min(length, x.shape[0] - first))
        return x[first:first + n], torch.ones(n, dtype=torch.bool)
    if x.dim() == 3:
        x = x[:, :, None]
    if layout == "BNBD":
        x = x.transpose(1, 2)
    n = min(length, block_table.shape[1] * P)
    rows = torch.zeros(n, x.shape[2], x.shape[3], dtype=x.dtype)
    there = torch.zeros(n, dtype=torch.bool)
    for i in range(-(-n // P)):
        page = int(block_table[b, i])
        m = min(P, n - i * P)
        if 0 <= page < x.shape[0]:
            rows[i * P:i * P + m] = x[page, :m]
            there[i * P:i * P + m] = True
    return rows, there


def attention(query, key, value, block_table, cu_seqlens_q, kv_len, layout, sparse_mode,
              scale: Optional[float] = None, blocks=None) -> Attention:
    T, Hq, _ = query.shape
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    spread = torch.zeros(T, Hq, D, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    size, top = (torch.zeros(T, Hq, dtype=torch.float64) for _ in range(2))
    count = torch.zeros(T, Hq, dtype=torch.int64)
    first = 0
    for b in range(len(kv_len)):
        length = max(int(kv_len[b]), 0)
        keys, there = request_rows(key, layout, block_table, b, length, first)
        vals, _ = request_rows(value, layout, block_table, b, length, first)
        first += length
        keys, vals = keys.double(), vals.double()
        g = Hq // keys.shape[1]
        j = torch.arange(keys.shape[0])
        for t, bt, pos in positions(cu_seqlens_q, kv_len, T):
            if bt != b:
                continue
            seen = there & (j <= pos) if sparse_mode == 3 else there
            for h in range(Hq):
                mine = seen
                if blocks is not None:
                    named = blocks[t, h // g]
                    mine = seen & torch.isin(j // P, named[named >= 0].long())
                if not bool(mine.any()):
                    continue
                k, v = keys[mine, h // g], vals[mine, h // g]
                q = query[t, h].double()
                s = scale * (k @ q)
                m = s.max()
                w = torch.exp(s - m)
                w = w / w.sum()
                out[t, h] = w @ v
                spread[t, h] = w @ v.abs()
                lse[t, h] = torch.logsumexp(s, 0)
                size[t, h] = (scale * (k.abs() @ q.abs())).max()
                count[t, h] = int(mine.sum())
                top[t, h] = v.abs().max()
    return Attention(out, lse, spread, size, count, top)


def attention_bounds(ref: Attention, dtype: torch.dtype):
    """(largest |out error| [T, Hq, D], largest |lse error| [T, Hq]) of an
    evaluation whose products accumulate in float32 and whose weights and
    result are rounded to ``dtype``.

    With e = 2^-24 and u = eps / 2 of the type, a score of 128 products is off
    by at most ds = 130 e size (128 additions, the scale, its constant) and
    its weight by the factor 1 +- (ds + 4 e (1 + size)) (the exponent's own
    rounding and exp2's); rounding it costs u more.  The smallest step of
    float16 is 2^-24; weights that are scaled so that the row's largest is at
    least 2^11 are off by half of that, 2^-36 of their sum (n of them: n 2^-36
    of the largest value).  The sums of n weights and products add n e each, a
    rescaling of the sums 2 e per 64 keys (within n e).  The quotient is off by
    both sums' shares, and u at its own rounding."""
    e = 2.0 ** -24
    u = torch.finfo(dtype).eps / 2
    n = ref.keys.double()
    dw = 130 * e * ref.size + 4 * e * (1 + ref.size)
    share = 2 * dw + 2 * n * e + 4 * e
    out = ref.spread * (share + u * (1 + share))[..., None] + u * ref.out.abs() * 1.01
    if dtype == torch.float16:
        out = out + (n * 2.0 ** -36 * ref.top)[..., None] + 2.0 ** -25
    lse = dw + n * e + 4 * e * (1 + ref.lse.abs().nan_to_num(0, 0, 0))
    return out, lse


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------


def rotated(x, cos, sin, interleaved: bool):
    """A row [128] rotated in binary64 by the angles [rotary / 2], and the sum
    of the magnitudes of the terms of each element."""
    y, mag = x.double().clone(), x.double().abs().clone()
    half = len(cos)
    for r in range(half):
        i, k = (2 * r, 2 * r + 1) if interleaved else (r, r + half)
        a, b, c, s = float(x[i]), float(x[k]), float(cos[r]), float(sin[r])
        y[i], y[k] = a * c - b * s, b * c + a * s
        mag[i], mag[k] = abs(a * c) + abs(b * s), abs(b * c) + abs(a * s)
    return y, mag


def encode_i8(y):
    """(codes [128] int8, scale float32)"""
    if not bool(torch.isfinite(y).all()):
        return torch.zeros(D, dtype=torch.int8), torch.tensor(math.nan)
    scale = (y.abs().max() / 127).to(torch.float32)
    if float(scale) == 0:
        return torch.zeros(D, dtype=torch.int8), scale
    return torch.tensor([max(-127, min(127, round(float(v) / float(scale)))) for v in y],
                        dtype=torch.int8), scale


def encode_fp8(y, dtype):
    """The nearest value of the format (ties to the even code), by search over
    all its finite codes; values past the largest stay at it."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    vals = codes.view(dtype).double()
    keep = torch.isfinite(vals) & (codes < 128)
    grid, names = vals[keep].sort()
    names = codes[keep][names]
    out = torch.zeros(D, dtype=torch.uint8)
    for i, v in enumerate(y.double()):
        if math.isnan(float(v)):
            out[i] = 0x7F
            continue
        d = (grid - min(abs(float(v)), float(grid[-1]))).abs()
        near = names[d == d.min()]
        code = int(min(near.tolist(), key=lambda n: n & 1))
        out[i] = code | (128 if math.copysign(1.0, float(v)) < 0 else 0)
    return out.view(dtype)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def encode_mxfp4(y):
    """(pairs [64] uint8, E8M0 [4] uint8)"""
    nib, scales = [], []
    for c in range(0, D, 32):
        g = y[c:c + 32]
        if not bool(torch.isfinite(g).all()):
            scales.append(255)
            nib += [0] * 32
            continue
        top = float(g.abs().max())
        e = 0 if top == 0 else max(0, min(254, math.frexp(top)[1] - 1 - 2 + 127))
        scales.append(e)
        for v in g.tolist():
            a = math.ldexp(abs(v), 127 - e)
            best = min(range(8), key=lambda i: (abs(min(a, 6.0) - _E2M1[i]), i & 1))
            nib.append(best | (8 if v < 0 and best else 0))
    return (torch.tensor([nib[i] | nib[i + 1] << 4 for i in range(0, D, 2)], dtype=torch.uint8),
            torch.tensor(scales, dtype=torch.uint8))


def append(item, cos, sin, block_table, cu_seqlens_q, kv_len, interleaved, any_rotated,
           axis_positions=None, pair_axes=None):
    """What ``msa_cache_append`` leaves of one item (src, dst, layout, scale,
    rotate; CPU tensors): (dst, scale, exact float64 rows, term magnitudes, written
    mask [T, H]), the rows and magnitudes per token and head.  With
    ``axis_positions`` [axes, T] pair r turns by the position of axis
    ``pair_axes[r]``."""
    src, dst, layout, scale, rotate = item
    T, H, _ = src.shape
    dst = dst.clone()
    scale = None if scale is None else scale.clone()
    rows = torch.zeros(T, H, D, dtype=torch.float64)
    mags = torch.zeros(T, H, D, dtype=torch.float64)
    written = torch.zeros(T, H, dtype=torch.bool)
    kv = [max(int(x), 0) for x in kv_len]
    for t, b, pos in positions(cu_seqlens_q, kv_len, T):
        turns = [pos] * (cos.shape[1] if any_rotated else 0)
        if any_rotated and axis_positions is not None:
            if not all(0 <= int(x) < cos.shape[0] for x in axis_positions[:, t]):
                continue
            turns = [int(axis_positions[a, t]) for a in pair_axes]
        if pos < 0 or (turns and max(turns) >= cos.shape[0]):
            continue
        pair = torch.arange(len(turns))
        for h in range(H):
            y, mag = src[t, h].double(), src[t, h].double().abs()
            if rotate:
                y, mag = rotated(src[t, h], cos[turns, pair], sin[turns, pair], interleaved)
            if layout == "ROWS":
                at, sat = (t, h), (t, h)
            elif layout == "TND":
                at = sat = (sum(kv[:b]) + pos, h)
                if at[0] >= dst.shape[0]:
                    continue
            else:
                blk = pos // P
                page = int(block_table[b, blk]) if blk < block_table.shape[1] else -1
                if not 0 <= page < dst.shape[0]:
                    continue
                at = (page, pos % P, h) if layout == "BBND" else (page, h, pos % P)
                if dst.dim() == 3:
                    at = at[:2]
                sat = (page, h, pos % P) if dst.dtype == torch.int8 else at
            rows[t, h], mags[t, h], written[t, h] = y, mag, True
            if dst.dtype == torch.int8:
                dst[at], scale[sat] = encode_i8(y)
            elif dst.dtype == torch.uint8:
                dst[at], scale[sat] = encode_mxfp4(y)
            elif dst.element_size() == 1:
                dst.view(torch.uint8)[at] = encode_fp8(y, dst.dtype).view(torch.uint8)
            else:
                dst[at] = y.float().to(dst.dtype)
    return dst, scale, rows, mags, written


# ---------------------------------------------------------------------------
# the step's tables
# ---------------------------------------------------------------------------


def step_tables(new_tokens, ctx_len, rows, pool, free_pages, free_count: int, max_blocks: int,
                T: int):
    """What ``msa_step_tables`` leaves, request by request: a dict of lists and
    tensors (``pool`` a changed copy, ``free`` the two counts)."""
    pool = pool.clone()
    B = len(new_tokens)
    count = min(max(int(free_count), 0), len(free_pages))
    stack = [int(x) for x in free_pages[:count]]
    missing = 0
    out = {"cu_seqlens_q": [0], "kv_len": [], "start_loc": [], "cu_pages": [0],
           "block_table": torch.full((B, max_blocks), -1, dtype=torch.int32),
           "positions": [], "slots": []}
    for b in range(B):
        q, c = max(int(new_tokens[b]), 0), max(int(ctx_len[b]), 0)
        row = b if rows is None else int(rows[b])
        held = 0 <= row < pool.shape[0]
        blocks = [-1] * max_blocks
        for k in range(min(max_blocks, -(-(c + q) // P))):
            if held and k >= -(-c // P):
                missing += not stack
                pool[row, k] = stack.pop() if stack else -1
            if held:
                blocks[k] = int(pool[row, k])
        out["block_table"][b] = torch.tensor(blocks, dtype=torch.int32)
        for pos in range(c, c + q):
            page = blocks[pos // P] if pos // P < max_blocks else -1
            out["positions"].append(pos)
            out["slots"].append(page * P + pos % P if page >= 0 else -1)
        out["cu_seqlens_q"].append(out["cu_seqlens_q"][-1] + q)
        out["kv_len"].append(c + q)
        out["start_loc"].append(c // P)
        out["cu_pages"].append(count - len(stack))
    pad = T - len(out["positions"])
    out["positions"] += [0] * pad
    out["slots"] += [-1] * pad
    return out | {"pool": pool, "free": [len(stack), missing]}


# ---------------------------------------------------------------------------
# attention with other forms of the scores
# ---------------------------------------------------------------------------


class Forms(NamedTuple):
    """Capped, biased, narrowed attention of every token, in binary64, with what
    its bounds take (all [T, Hq] but the first, the third and the fourth)."""
    out: torch.Tensor      # [T, Hq, D]
    lse: torch.Tensor
    spread: torch.Tensor   # [T, Hq, D]: sum of |weight * value|
    drift: torch.Tensor    # [T, Hq, D]: sum of |weight's error * value|
    loss: torch.Tensor     # sum of the weights' errors
    keys: torch.Tensor     # visible keys
    top: torch.Tensor      # largest |value| of a visible key
    shift: torch.Tensor    # |bias| of the nearest key in the token's range


def attention_forms(query, key, value, block_table, cu_seqlens_q, kv_len, layout, sparse_mode,
                    scale: Optional[float] = None, softcap: float = 0.0, slopes=None,
                    visible=None) -> Forms:
    """``msa_attention_ex`` from its definition, a request and a head at a time.

    A weight's error, with e = 2^-24: the product of 128 terms is off by at most
    130 e of its size (the sum of its terms' magnitudes and, as the sums may begin
    with it, the bias), the cap by 12 e of softcap (exponential, sum, reciprocal,
    product: 10 e; the polynomial 4.5 e and its own 6 roundings of at most 0.75
    softcap), the bias by 2 e, and the exponent by 4 e (1 + |S2| + max |S2|); the
    weight exp(S2) then changes by the factor exp(+-d).  Where the errors add up to
    more than all weights (scores of 10^7 and more), the result is still a mean of
    visible values, off by twice the largest of them at most, and the log of the sum
    by the largest d."""
    T, Hq, _ = query.shape
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    e = 2.0 ** -24
    f = Forms(*(torch.zeros(T, Hq, *([D] if i in (0, 2, 3) else []), dtype=torch.float64)
                for i in range(8)))
    f.lse.fill_(-math.inf)
    first = 0
    cu = [int(x) for x in cu_seqlens_q]
    for b in range(len(kv_len)):
        length = max(int(kv_len[b]), 0)
        keys, there = request_rows(key, layout, block_table, b, length, first)
        vals, _ = request_rows(value, layout, block_table, b, length, first)
        first += length
        lo, hi = max(cu[b], 0), min(cu[b + 1], T)
        if hi <= lo or not len(keys):
            continue
        pos = (int(kv_len[b]) - (cu[b + 1] - cu[b]) + torch.arange(lo, hi) - cu[b])[:, None]
        j = torch.arange(keys.shape[0])[None]
        inside = torch.ones(hi - lo, keys.shape[0], dtype=torch.bool)
        if sparse_mode == 3:
            inside = inside & (j <= pos)
        if visible is not None:
            span = visible[lo:hi].long()
            inside = inside & (j >= span[:, :1]) & (j < span[:, 1:])
        seen = inside & there[None]
        away = (pos - j).abs().double()
        least = torch.where(inside, away, math.inf).amin(1, keepdim=True).nan_to_num(0, 0, 0)
        g = Hq // keys.shape[1]
        some = seen.any(1)
        kd, qd = keys[there].double(), query[lo:hi].double()
        near = bool(softcap) and all(
            bool((scale * (qd[:, h] @ kd[:, h // g].T).abs() <= 0.62 * softcap).all())
            for h in range(Hq))
        for h in range(Hq):
            k, v, q = keys[:, h // g].double(), vals[:, h // g].double(), query[lo:hi, h].double()
            s = scale * (q @ k.T)
            d = 130 * e * scale * (q.abs() @ k.abs().T)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                d = d + (8 * e * s.abs() if near else 12 * e * softcap)
            base = 0.0
            if slopes is not None:
                bias, base = float(slopes[h]) * (away - least), float(slopes[h]) * least
                d = d + (0 if softcap else 130 * e) * bias.abs() + 2 * e * bias.abs()
                s = s - bias
                f.shift[lo:hi, h] = base[:, 0].abs()
            s = torch.where(seen, s, -math.inf)
            m = torch.where(some, s.amax(1), 0.0)[:, None]
            d = d + 4 * e * (1 + torch.where(seen, s, 0.0).abs() + m.abs())
            w = torch.where(seen, torch.exp(s - m), 0.0)
            w = w / torch.where(some, w.sum(1), 1.0)[:, None]
            off = torch.where(seen, w * torch.expm1(d), 0.0)
            v = torch.where(seen.any(0)[:, None], v, 0.0)
            f.out[lo:hi, h] = w @ v
            f.spread[lo:hi, h] = w @ v.abs()
            big = torch.where(seen, v.abs().amax(1)[None], 0.0).amax(1)
            loss = off.sum(1)
            wild = ~(loss <= 1)          # (0 * inf among them)
            f.drift[lo:hi, h] = torch.where(wild[:, None], 2 * big[:, None], off @ v.abs())
            f.loss[lo:hi, h] = torch.where(wild, torch.where(seen, d, 0.0).amax(1), loss)
            f.lse[lo:hi, h] = torch.logsumexp(s - base, 1)
            f.keys[lo:hi, h] = seen.sum(1).double()
            f.top[lo:hi, h] = big
    return f


def forms_bounds(f: Forms, dtype: torch.dtype):
    """(largest |out error| [T, Hq, D], largest |lse error| [T, Hq]), as
    ``attention_bounds``: the weights' errors, n e for each of the two sums of n
    terms and as much for their rescalings, half a step for a weight and for the
    result, and float16's smallest step."""
    e = 2.0 ** -24
    u = torch.finfo(dtype).eps / 2
    share = 2 * f.keys * e + 4 * e
    out = (1.01 * (f.drift + f.spread * f.loss[..., None])
           + f.spread * (share + u * (1.01 + f.loss))[..., None] + u * f.out.abs() * 1.01)
    if dtype == torch.float16:
        out = out + (f.keys * 2.0 ** -36 * f.top)[..., None] + 2.0 ** -25
    lse = (1.01 * f.loss + f.keys * e + 4 * e * (1 + f.lse.abs().nan_to_num(0, 0, 0))
           + 4 * e * f.shift)
    return out, lse
