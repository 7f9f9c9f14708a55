"""The cache append against the oracle (oracle/layer.py): 16-bit rows within a
half step of the binary64 rotation (and the float32 evaluation's own error),
encoded rows bit for bit, and every place that no row goes to as it was."""
import sys

import pytest
import torch

import layer_cases as lc
from oracle import layer

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
KINDS = {"same": None, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "i8": torch.int8,
         "mxfp4": torch.uint8}


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_max_qk_amd
    block_max_qk_amd.load_library()
    return torch.device("cuda:0")


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def angles(n, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n, dtype=torch.float64)[:, None] * inv
    return a.cos().float(), a.sin().float()


def make_item(src, kind, layout, T, H, pages, n_keys, gen, rotate):
    """(src, dst, layout, scale, rotate) with a destination full of old values."""
    dt = KINDS[kind] or src.dtype
    last = 64 if kind == "mxfp4" else 128
    lead = {"ROWS": (T, H), "TND": (n_keys, H)}.get(layout)
    shape = (*lead, last) if lead else lc.cache_shape(layout, pages, H, last)
    n = 1
    for x in shape:
        n *= x
    old = torch.randint(0, 100, (n,), generator=gen, dtype=torch.int32)
    dst = old.to(dt).view(shape) if dt in (torch.int8, torch.uint8) else old.float().to(dt).view(shape)
    scale = None
    if kind == "i8":
        scale = torch.full((*lead,) if lead else (pages, H, 128), 7.0)
    elif kind == "mxfp4":
        scale = torch.full((*shape[:-1], 4), 9, dtype=torch.uint8)
    return [src, dst, layout, scale, rotate]


def batch(q_lens, kv_lens, seed, width=None, T_extra=0, first=0):
    gen = torch.Generator().manual_seed(seed)
    cu, T = lc.lengths(q_lens, T_extra, first)
    table, pages = lc.table_for(kv_lens, gen, width=width)
    return gen, cu, T, torch.tensor(kv_lens, dtype=torch.int32), table, pages


def run(items, cos, sin, table, cu, kv, dev, interleaved=False, srcs=None, **kw):
    """Call on the device; compare every item with the oracle."""
    import block_max_qk_amd as m
    put = lambda x: None if x is None else x.to(dev)  # noqa: E731
    live = [m.CacheItem(put(i[0]) if srcs is None else srcs[k], put(i[1]), i[2], put(i[3]), i[4])
            for k, i in enumerate(items)]
    m.msa_cache_append(live, put(cos), put(sin), put(table), put(cu), put(kv),
                       interleaved=interleaved, **kw)
    torch.cuda.synchronize()
    rotated = any(i[4] for i in items)
    for i, d in zip(items, live):
        dst, scale, rows, mags, written = layer.append(i, cos, sin, table, cu, kv, interleaved,
                                                       rotated)
        got = d.dst.cpu()
        if i[1].element_size() == 1:
            # (a format has several codes that are NaN: any of them will do)
            nan = torch.isnan(dst.float()) if i[1].dtype.is_floating_point else torch.zeros(1) > 0
            assert torch.equal(torch.isnan(got.float()), torch.isnan(dst.float()))
            wrong = ((bits(got) != bits(dst)) & ~nan).nonzero()
            assert not len(wrong), (i[2], i[1].dtype, wrong[:4].tolist())
            if scale is not None:
                gs = d.scale.cpu()
                nan = torch.isnan(scale.float())
                assert torch.equal(torch.isnan(gs.float()), nan)
                assert torch.equal(bits(gs)[~nan], bits(scale)[~nan])
            continue
        if not i[4]:
            assert torch.equal(bits(got), bits(dst))
            continue
        # every place that differs from the oracle's holds a row, and is within
        # half a step (of the value as evaluated) and three float32 roundings
        # (two products, one sum) of the binary64 value
        info = torch.finfo(got.dtype)
        err = (got.double() - exact_dst(i, rows, written, table, cu, kv, cos)).abs()
        near = exact_dst(i, mags, written, table, cu, kv, cos) * 3 * 2.0 ** -24
        tol = near + (dst.double().abs() + near) * info.eps / 2 * 1.01 + info.smallest_normal * info.eps
        same = bits(got) == bits(dst)
        assert (same | (err <= tol)).all(), float((err / tol)[~same].max())
        # (a float32 evaluation lands on another 16-bit value than the oracle's
        # only next to a border: rarely)
        assert (~same).float().mean() < 0.02
    return live


def exact_dst(i, rows, written, table, cu, kv, cos):
    """The destination in float64 with the given rows in their places."""
    src, dst, layout, _, _ = i
    full = dst.double().clone()
    lens = [max(int(x), 0) for x in kv]
    for t, b, pos in layer.positions(cu, kv, src.shape[0]):
        for h in range(src.shape[1]):
            if not written[t, h]:
                continue
            if layout == "ROWS":
                full[t, h] = rows[t, h]
            elif layout == "TND":
                full[sum(lens[:b]) + pos, h] = rows[t, h]
            else:
                page = int(table[b, pos // 128])
                if layout == "BBND":
                    full[page, pos % 128, h] = rows[t, h]
                else:
                    full[page, h, pos % 128] = rows[t, h]
    return full


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("layout", ["BBND", "BNBD", "TND", "ROWS"])
@pytest.mark.parametrize("pairs", ["halves", "interleaved"])
def test_kinds_and_layouts(dtype, kind, layout, pairs, dev):
    log("append", dtype, kind, layout, pairs)
    q_lens, kv_lens = [1, 7, 0, 4], [1, 135, 50, 4]
    gen, cu, T, kv, table, pages = batch(q_lens, kv_lens, 40)
    cos, sin = angles(140, 128)
    src = torch.randn(T, 3, 128, generator=gen).to(dtype)
    items = [make_item(src, kind, layout, T, 3, pages, sum(kv_lens), gen, r) for r in (True, False)]
    run(items, cos, sin, table, cu, kv, dev, pairs == "interleaved")


@pytest.mark.parametrize("rot", [16, 32, 48, 64, 96, 128])
@pytest.mark.parametrize("pairs", ["halves", "interleaved"])
def test_rotated_part(rot, pairs, dev):
    gen, cu, T, kv, table, pages = batch([3, 2], [260, 2], 41)
    cos, sin = angles(260, rot)
    src = torch.randn(T, 5, 128, generator=gen).to(BF)
    items = [make_item(src, kind, "BBND", T, 5, pages, 0, gen, True) for kind in KINDS]
    run(items, cos, sin, table, cu, kv, dev, pairs == "interleaved")


def test_a_layers_items_in_one_call(dev):
    """Queries, keys, values and both index rows, of different head counts,
    the sources side by side in wider rows."""
    gen, cu, T, kv, table, pages = batch([1, 20, 3], [129, 20, 300], 42)
    cos, sin = angles(300, 64)
    qkv = torch.randn(T, 24, 128, generator=gen).to(BF)
    iqk = torch.randn(T, 5, 128, generator=gen).to(BF)
    parts = [(qkv[:, :16], "same", "ROWS", True), (qkv[:, 16:20], "same", "BNBD", True),
             (qkv[:, 20:], "same", "BNBD", False), (iqk[:, :4], "mxfp4", "ROWS", True),
             (iqk[:, 4:], "mxfp4", "BNBD", True)]
    items = [make_item(s, k, lay, T, s.shape[1], pages, 0, gen, r) for s, k, lay, r in parts]
    a, b = qkv.to(dev), iqk.to(dev)
    srcs = [a[:, :16], a[:, 16:20], a[:, 20:], b[:, :4], b[:, 4:]]
    run(items, cos, sin, table, cu, kv, dev, srcs=srcs)


def test_many_tokens(dev):
    """Long runs: several steps a wave, more requests than one search step."""
    gen = torch.Generator().manual_seed(43)
    q = torch.randint(0, 9, (130,), generator=gen).tolist()
    kv_lens = [n + int(x) for n, x in zip(q, torch.randint(0, 90, (130,), generator=gen))]
    gen, cu, T, kv, table, pages = batch(q, kv_lens, 44)
    cos, sin = angles(100, 128)
    for layout in ("BBND", "TND"):
        src = torch.randn(T, 70, 128, generator=gen).to(FP)
        run([make_item(src, "same", layout, T, 70, pages, sum(kv_lens), gen, False),
             make_item(src[:, :1], "i8", layout, T, 1, pages, sum(kv_lens), gen, True)],
            cos, sin, table, cu, kv, dev)


def test_long_runs_of_tokens(dev):
    """A chunk long enough for the launch's longest wave runs."""
    gen, cu, T, kv, table, pages = batch([4000], [4000], 45)
    cos, sin = angles(4000, 128)
    src = torch.randn(T, 90, 128, generator=gen).to(BF)
    items = [make_item(src, "same", "BBND", T, 90, pages, 0, gen, False)]
    import block_max_qk_amd as m
    live = m.CacheItem(src.to(dev), items[0][1].to(dev), "BBND")
    rot = torch.empty(T, 90, 128, dtype=BF, device=dev)
    m.msa_cache_append([live, m.CacheItem(live.src, rot, "ROWS", rotate=True)], cos.to(dev),
                       sin.to(dev), table.to(dev), cu.to(dev), kv.to(dev))
    torch.cuda.synchronize()
    pos = torch.arange(4000)
    want = items[0][1].clone()
    want[table[0, pos // 128].long(), pos % 128] = src
    assert torch.equal(bits(live.dst.cpu()), bits(want))
    x = src.double()
    c, s = cos.double()[:, None], sin.double()[:, None]
    y = torch.cat([x[..., :64] * c - x[..., 64:] * s, x[..., 64:] * c + x[..., :64] * s], -1)
    mag = torch.cat([(x[..., :64] * c).abs() + (x[..., 64:] * s).abs(),
                     (x[..., 64:] * c).abs() + (x[..., :64] * s).abs()], -1)
    near = 3 * 2.0 ** -24 * mag
    assert ((rot.cpu().double() - y).abs() <= near + (y.abs() + near) * 2.0 ** -8).all()


def test_tokens_that_are_skipped(dev):
    """Before position 0, past the angle table, on no page, behind the table,
    behind the last request: nothing is written."""
    gen, cu, T, kv, table, pages = batch([4, 3, 5, 2], [2, 300, 200, 256], 46, T_extra=6, first=2)
    table[1, 2] = -1                       # the page of positions 256 .. 299
    table[2, 1] = pages                    # of positions 128 .. 199
    kv[3] = 400                            # past the table's 3 blocks
    cos, sin = angles(299, 128)            # position 299 has no angles
    src = torch.randn(T, 2, 128, generator=gen).to(BF)
    for layout in ("BBND", "BNBD", "ROWS"):
        items = [make_item(src, kind, layout, T, 2, pages, 0, gen, True) for kind in KINDS]
        run(items, cos, sin, table, cu, kv, dev)
    gen, cu, T, kv, table, pages = batch([4, 3], [2, 30], 47, T_extra=6)
    items = [make_item(src[:T], kind, "TND", T, 2, pages, 30, gen, True) for kind in KINDS]
    run(items, cos, sin, table, cu, kv, dev)        # the tensor holds 30 of 32 keys


def test_values_at_the_encodings_edges(dev):
    """Ties, overflow, zero rows, subnormals, infinities and NaN."""
    gen, cu, T, kv, table, pages = batch([12], [12], 48)
    src = torch.randn(T, 2, 128, generator=gen)
    src[0] = 0
    src[1, 0] = torch.arange(128) / 16.0                       # ties of every format
    src[1, 1] = torch.arange(-64, 64) * 7.0
    src[2] *= 60000.0
    src[3] *= 1e-7
    src[4, 0, 5] = float("nan")
    src[5, 1, 77] = float("inf")
    src[6, 0, 3] = float("-inf")
    src[7] = 448.0
    src[8, :, ::2] = -0.0
    src[9] = torch.where(torch.rand(2, 128, generator=gen) < 0.5, 6.0, 0.25)
    src[10] = 464.0
    for dtype in (BF, FP):
        items = [make_item(src.to(dtype), kind, "BBND", T, 2, pages, 0, gen, False)
                 for kind in KINDS]
        run(items, None, None, table, cu, kv, dev)


def test_rotation_in_place(dev):
    """The queries' rows may be rotated where they are."""
    import block_max_qk_amd as m
    gen, cu, T, kv, table, pages = batch([9, 40], [9, 77], 49)
    cos, sin = angles(80, 128)
    q = torch.randn(T, 16, 128, generator=gen).to(BF).to(dev)
    other = torch.empty_like(q)
    args = (cos.to(dev), sin.to(dev), None, cu.to(dev), kv.to(dev))
    m.msa_cache_append([m.CacheItem(q, other, "ROWS", rotate=True)], *args)
    m.msa_cache_append([m.CacheItem(q, q, "ROWS", rotate=True)], *args)
    torch.cuda.synchronize()
    assert torch.equal(q, other)


def test_strided_destinations(dev):
    """Pages with gaps, rows in wider rows; what lies between stays."""
    import block_max_qk_amd as m
    gen, cu, T, kv, table, pages = batch([5, 3], [133, 3], 50)
    src = torch.randn(T, 2, 128, generator=gen).to(FP)
    wide = torch.full((pages, 2, 128, 2, 128), 5.0, dtype=FP, device=dev)
    rows = torch.full((T, 7, 128), 6.0, dtype=FP, device=dev)
    flat = torch.empty(pages, 128, 2, 128, dtype=FP, device=dev).fill_(5.0)
    args = (None, None, table.to(dev), cu.to(dev), kv.to(dev))
    s = src.to(dev)
    m.msa_cache_append([m.CacheItem(s, wide[:, 1], "BBND"), m.CacheItem(s, flat, "BBND"),
                        m.CacheItem(s, rows[:, 3:5], "ROWS")], *args)
    torch.cuda.synchronize()
    assert (wide[:, 0] == 5).all() and torch.equal(wide[:, 1], flat)
    assert (rows[:, :3] == 6).all() and (rows[:, 5:] == 6).all()
    assert torch.equal(rows[:, 3:5], s)
