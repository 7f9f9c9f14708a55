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


def append(item, cos, sin, block_table, cu_seqlens_q, kv_len, interleaved, any_rotated):
    """What ``msa_cache_append`` leaves of one item (src, dst, layout, scale,
    rotate; CPU tensors): (dst, scale, exact float64 rows, term magnitudes, written
    mask [T, H]), the rows and magnitudes per token and head."""
    src, dst, layout, scale, rotate = item
    T, H, _ = src.shape
    dst = dst.clone()
    scale = None if scale is None else scale.clone()
    rows = torch.zeros(T, H, D, dtype=torch.float64)
    mags = torch.zeros(T, H, D, dtype=torch.float64)
    written = torch.zeros(T, H, dtype=torch.bool)
    kv = [max(int(x), 0) for x in kv_len]
    for t, b, pos in positions(cu_seqlens_q, kv_len, T):
        if pos < 0 or (any_rotated and pos >= cos.shape[0]):
            continue
        for h in range(H):
            y, mag = src[t, h].double(), src[t, h].double().abs()
            if rotate:
                y, mag = rotated(src[t, h], cos[pos], sin[pos], interleaved)
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
