"""Attention with capped scores, a bias by distance and a visible range per token
against the binary64 oracle (oracle/layer.py), within bounds derived from the
arithmetic (``forms_bounds`` there), through each kernel: 16-row tiles, 128- and
256-row tiles, with and without a split over the keys."""
import ctypes
import sys

import pytest
import torch

import layer_cases as lc
from oracle import layer

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_max_qk_amd
    block_max_qk_amd.load_library()
    return torch.device("cuda:0")


def pos_of(c):
    pos = torch.zeros(c["q"].shape[0], dtype=torch.int64)
    for t, _, x in layer.positions(c["cu"], c["kv"], len(pos)):
        pos[t] = x
    return pos


def spans(c, kind, seed=0):
    """Ranges of the case's tokens: documents (mode 3), images or a prefix (mode
    0), or any ranges at all."""
    gen = torch.Generator().manual_seed(seed)
    pos = pos_of(c)
    top = int(max(c["kv"].max(), 1))
    if kind == "documents":
        size = max(1, top // 4)
        return torch.stack([pos // size * size, pos // size * size + size], 1).int()
    if kind == "images":
        size = max(1, top // 5)
        image = pos // size % 2 == 1
        end = torch.where(image, pos // size * size + size, pos + 1)
        return torch.stack([torch.zeros_like(pos), end], 1).int()
    if kind == "prefix":
        return torch.stack([torch.zeros_like(pos), (pos + 1).clamp(min=top // 2)], 1).int()
    a = torch.randint(-20, top + 20, (len(pos), 2), generator=gen)
    return a.int()


def make(q_lens, kv_lens, Hq, Hkv, layout="BBND", dtype=BF, mode=3, cap=0.0, bias=False,
         mask=None, gain=3.0, seed=0, **kw):
    c = lc.attention_case(q_lens, kv_lens, Hq, Hkv, layout, dtype, mode, seed, **kw)
    c["q"] = (c["q"].float() * gain).to(dtype)
    c["cap"] = cap
    c["slopes"] = (2.0 ** (-8 * torch.arange(1, Hq + 1) / Hq)).float() if bias else None
    c["visible"] = spans(c, mask, seed) if mask else None
    return c


def call(c, dev, **kw):
    import block_max_qk_amd as m
    d = {n: (x.to(dev) if torch.is_tensor(x) else x) for n, x in c.items()}
    q = d["q"]
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=dev)
    lse = torch.full(q.shape[:2], float("nan"), device=dev)
    mb = d["table"].shape[1] if d["table"] is not None else (d["k"].shape[0] + 127) // 128
    m.msa_attention(q, d["k"], d["v"], d["table"], d["cu"], d["kv"], d["layout"], d["mode"],
                    d.get("scale"), out, mb, lse=lse, softcap=d["cap"], slopes=d["slopes"],
                    visible=d["visible"], **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def reference(c):
    return layer.attention_forms(c["q"], c["k"], c["v"], c["table"], c["cu"], c["kv"],
                                 c["layout"], c["mode"], c.get("scale"), c["cap"], c["slopes"],
                                 c["visible"])


def check(c, out, lse, ref=None):
    ref = reference(c) if ref is None else ref
    first, end = int(c["cu"][0]), int(c["cu"][-1])
    tol_out, tol_lse = (x[first:end] for x in layer.forms_bounds(ref, c["q"].dtype))
    ref = layer.Forms(*(x[first:end] for x in ref))
    out, lse = out.double()[first:end], lse.double()[first:end]
    assert torch.isfinite(out).all()
    err = (out - ref.out).abs()
    assert (err <= tol_out).all(), float((err / tol_out.clamp(min=1e-30)).max())
    empty = ref.keys == 0
    assert (out[empty] == 0).all()
    assert torch.equal(lse == -torch.inf, empty)
    err = (lse - ref.lse).abs()[~empty]
    assert (err <= tol_lse[~empty]).all(), float((err / tol_lse[~empty]).max())


def run(c, dev, **kw):
    check(c, *call(c, dev, **kw))


FORMS = [dict(cap=30.0), dict(bias=True), dict(cap=20.0, bias=True), dict(mask="documents"),
         dict(cap=5.0, mask="any"), dict(bias=True, mask="any"),
         dict(cap=50.0, bias=True, mask="documents"), dict(mode=0, mask="images", cap=30.0),
         dict(mode=0, mask="prefix", bias=True), dict(mode=0, bias=True)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("layout", ["BBND", "BNBD", "TND"])
def test_decode(form, layout, dtype, dev):
    """Single tokens, 16-row tiles, groups of one head to more than a tile."""
    for Hq, Hkv in ((1, 1), (10, 2), (40, 2)):
        log("decode", form, layout, dtype, Hq, Hkv)
        run(make([1, 1, 0, 1, 1], [1, 127, 300, 128, 577], Hq, Hkv, layout, dtype, seed=Hq,
                 **form), dev)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,layout,dtype", [
    ([33], [33], 8, 2, "TND", BF), ([70, 1, 9], [70, 300, 129], 6, 2, "BNBD", FP),
    ([129], [260], 4, 4, "BBND", FP), ([17, 40], [65, 104], 24, 1, "TND", FP),
    ([5], [700], 300, 1, "BBND", BF), ([2, 3], [200, 131], 8, 1, "BBND", BF),
])
def test_chunks(form, q_lens, kv_lens, Hq, Hkv, layout, dtype, dev):
    log("chunks", form, q_lens, Hq, Hkv, layout, dtype)
    run(make(q_lens, kv_lens, Hq, Hkv, layout, dtype, seed=sum(q_lens), **form), dev)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_many_rows(form, dtype, dev):
    """Tiles of 256 rows, ragged ends of tiles and stages."""
    import block_max_qk_amd as m
    c = make([515, 301], [515, 430], 32, 8, "BBND", dtype, seed=5, **form)
    assert m.msa_attention_tile_rows(816, 2, 32, 8, c["table"].shape[1]) in (128, 256)
    log("many rows", form, dtype)
    run(c, dev)


def test_256_row_tiles(dev):
    import block_max_qk_amd as m
    for form in FORMS:
        for width in (17, 130):          # (256 rows only in tables of 128 blocks and more)
            c = make([700, 900], [700, 2100], 32, 16, "BBND", BF, seed=8, width=width, **form)
            assert m.msa_attention_tile_rows(1600, 2, 32, 16, width) == 256
            log("256", form, width)
            run(c, dev)


@pytest.mark.parametrize("form", FORMS)
def test_split_over_keys(form, dev):
    import block_max_qk_amd as m
    for q_lens, kv_lens, Hq, Hkv in (([1, 1], [5000, 129], 16, 2), ([40], [3333], 16, 2),
                                     ([2, 50, 1], [3000, 2500, 77], 8, 2)):
        c = make(q_lens, kv_lens, Hq, Hkv, seed=len(q_lens), **form)
        assert m.msa_attention_workspace(sum(q_lens), len(q_lens), Hq, Hkv,
                                         c["table"].shape[1]) > 0
        log("split", form, q_lens)
        run(c, dev)


@pytest.mark.parametrize("q_lens,kv_lens", [([7, 1], [300, 129]), ([90], [400]), ([1], [2000])])
def test_odd_ranges(q_lens, kv_lens, dev):
    """Ranges that are empty, turned round, outside the keys, of one key, and of
    the largest and smallest numbers; and tokens that all see nothing."""
    big, low = 2 ** 31 - 1, -2 ** 31
    picks = [(0, 0), (5, 2), (low, low), (big, big), (low, big), (big, low), (0, 1), (127, 129),
             (128, 129), (0, big), (63, 64), (200, 1 << 20), (-1, 5)]
    for mode in (0, 3):
        for bias in (False, True):
            c = make(q_lens, kv_lens, 4, 2, mode=mode, bias=bias, cap=0.0)
            T = c["q"].shape[0]
            for shift in range(3):
                c["visible"] = torch.tensor([picks[(5 * t + shift) % len(picks)]
                                             for t in range(T)], dtype=torch.int32)
                run(c, dev)
            c["visible"] = torch.zeros(T, 2, dtype=torch.int32)
            run(c, dev)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv", [([1], [300], 4, 1), ([5, 1], [290, 140], 4, 2),
                                                   ([100], [300], 8, 2), ([600], [600], 32, 16)])
def test_unseen_values_stay_away(bad, q_lens, kv_lens, Hq, Hkv, dev):
    """Keys and values that no row, or only other rows of a tile, see may be
    infinite or NaN: a row's result is that of clean ones."""
    for form in (dict(cap=30.0), dict(bias=True), dict(cap=9.0, bias=True), dict()):
        c = make(q_lens, kv_lens, Hq, Hkv, "TND", BF, **form)
        pos = pos_of(c)
        # each token sees 21 keys up to its own; of each request, the key before
        # the last token's first one turns bad, which earlier tokens see, and key 0
        c["visible"] = torch.stack([(pos - 20).clamp(min=0), pos + 1], 1).int()
        want = reference(c)
        ok = torch.ones(len(pos), dtype=torch.bool)
        at = 0
        for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
            for j in {kv - 22, 0}:
                c["k"][at + j] = bad
                c["v"][at + j] = bad
                mine = slice(int(c["cu"][b]), int(c["cu"][b + 1]))
                ok[mine] &= (j < c["visible"][mine, 0]) | (j >= c["visible"][mine, 1])
            at += kv
        assert ok.any()
        out, lse = call(c, dev)
        tol_out, tol_lse = layer.forms_bounds(want, BF)
        assert ((out.double() - want.out).abs() <= tol_out)[ok].all(), (form, q_lens)
        assert ((lse.double() - want.lse).abs() <= tol_lse)[ok].all(), (form, q_lens)


def test_caps(dev):
    """Scores far past the cap, far below it, at it, and of both kinds in a tile."""
    for cap in (1e-3, 0.5, 8.0, 1e4, 1e30):
        for gain in (0.01, 3.0, 40.0):
            for q_lens, kv_lens in (([1, 2], [200, 130]), ([60], [200])):
                run(make(q_lens, kv_lens, 8, 2, cap=cap, gain=gain), dev)
    c = make([50], [300], 8, 2, cap=20.0)
    c["q"][10:20] *= 30
    c["q"][30:40] = 0
    run(c, dev)
    # scores that are infinite: the cap's ends
    c = make([3, 40], [100, 120], 4, 2, "TND", BF, cap=6.0)
    c["k"][50], c["k"][150] = 3e38, -3e38
    c["q"] = c["q"].abs().clamp(min=1.0)
    out, lse = call(c, dev)
    d = {**c, "k": c["k"].clone()}
    d["k"][50], d["k"][150] = 300.0, -300.0      # (the cap's ends too)
    check(d, out, lse)


def test_large_caps(dev):
    """Scores that come near caps of any size."""
    for cap in (1e5, 1e7, 1e12, 1e20, 1e30):
        for part in (0.02, 0.2, 0.7):
            for q_lens, kv_lens in (([1, 2], [200, 130]), ([60], [200])):
                c = make(q_lens, kv_lens, 8, 2, gain=1.0)
                top = reference({**c, "cap": 0.0}).lse.max()
                c["q"] = (c["q"].float() * float(part * cap / top)).to(BF)
                c["cap"] = cap
                run(c, dev)


def test_slopes(dev):
    """Zero, negative and steep ones; positions before 0 (more new tokens than
    keys) without a causal mask."""
    for mode in (0, 3):
        c = make([1, 30], [900, 200], 8, 2, mode=mode, bias=True)
        c["slopes"] = torch.tensor([0.0, -0.01, 4.0, 100.0, 1e-6, 0.5, -0.0, 0.1])
        run(c, dev)
        c = make([9, 200], [4, 150], 8, 2, mode=mode, bias=True)
        run(c, dev)


def test_scale_and_padding(dev):
    """A scale of its own; rows before the first and behind the last request stay
    as they were, whatever their ranges say."""
    c = make([3, 60], [50, 70], 8, 2, cap=10.0, bias=True, mask="any", T_extra=7, first=2)
    c["scale"] = 0.3
    out, lse = call(c, dev)
    check(c, out, lse)
    assert out[:2].isnan().all() and out[65:].isnan().all()
    assert lse[:2].isnan().all() and lse[65:].isnan().all()


def test_pages_that_are_missing(dev):
    for q_lens in ([1, 1], [30, 40]):
        c = make(q_lens, [500, 300], 8, 2, "BNBD", FP, cap=20.0, bias=True, mask="any")
        c["table"][0, 1] = -1
        c["table"][1, 2] = 10 ** 6
        run(c, dev)


def test_none_of_the_forms_is_the_plain_call(dev):
    """msa_attention_ex without cap, slopes and ranges: the same bits."""
    import block_max_qk_amd as m
    from block_max_qk_amd._binding import _packed
    for q_lens, kv_lens in (([1, 1], [700, 20]), ([100], [200])):
        c = {n: (x.to(dev) if torch.is_tensor(x) else x)
             for n, x in lc.attention_case(q_lens, kv_lens, 8, 2).items()}
        want, want_lse = m.attention(c["q"], c["k"], c["v"], c["table"], c["cu"], c["kv"], "BBND",
                                     return_lse=True)
        out, lse = torch.empty_like(want), torch.empty_like(want_lse)
        T, B, mb = sum(q_lens), len(q_lens), c["table"].shape[1]
        ws = torch.empty(m.msa_attention_workspace(T, B, 8, 2, mb) + 16, dtype=torch.uint8,
                         device=dev)
        st = m.load_library().msa_attention_ex(
            _packed(c["q"]), _packed(c["k"]), _packed(c["v"]), c["table"].data_ptr(), mb,
            c["cu"].data_ptr(), c["kv"].data_ptr(), B, 128, 1, 3, 128 ** -0.5, 0.0, None, None,
            out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
            ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream))
        assert st == 0
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("form", [dict(cap=20.0), dict(bias=True, mask="any"),
                                  dict(mask="documents")])
def test_workspaces_of_any_size(form, dev):
    """A call is split into as many parts as its workspace holds."""
    import block_max_qk_amd as m
    for q_lens, kv_lens in (([50], [2992]), ([40, 2, 9], [1500, 2300, 128]), ([33], [700]),
                            ([150, 90], [1100, 90]), ([900], [1000]), ([1, 1], [3000, 200])):
        c = make(q_lens, kv_lens, 16, 2, "BNBD", BF, seed=7, **form)
        T, B, mb = sum(q_lens), len(q_lens), c["table"].shape[1]
        row = T * 16 * (128 * 4 + 8)
        least = m.msa_attention_workspace(T, B, 16, 2, mb)
        most = m.msa_attention_ex_workspace(T, B, 16, 2, mb)
        ref = reference(c)
        for size in sorted({least, least + row, (least + most) // 2 // row * row + 48, most,
                            most + 5 * row}):
            if size < least:
                continue
            log("workspace", form, q_lens, size // row)
            # (bytes past the size that is given stay as they are)
            ws = torch.full((size + 256,), 77, dtype=torch.uint8, device=dev)
            check(c, *call(c, dev, workspace=ws[:size]), ref)
            assert (ws[size:] == 77).all()


def test_same_bits_again_and_on_a_stream(dev):
    import block_max_qk_amd as m
    for q_lens, kv_lens in (([1, 1], [3000, 20]), ([100], [2000])):
        c = make(q_lens, kv_lens, 8, 2, cap=20.0, bias=True, mask="documents")
        d = {n: (x.to(dev) if torch.is_tensor(x) else x) for n, x in c.items()}
        args = (d["q"], d["k"], d["v"], d["table"], d["cu"], d["kv"], "BBND")
        kw = dict(softcap=20.0, slopes=d["slopes"], visible=d["visible"], return_lse=True)
        a = m.attention(*args, **kw)
        side = torch.cuda.Stream(dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        b = m.attention(*args, stream=side, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_and_replayed(dev):
    """Slopes, ranges and lengths are read by each replay."""
    import block_max_qk_amd as m
    c = make([1, 1, 1], [2500, 300, 77], 16, 2, cap=20.0, bias=True, mask="any")
    d = {n: (x.to(dev) if torch.is_tensor(x) else x) for n, x in c.items()}
    out = torch.zeros_like(d["q"])
    lse = torch.zeros(d["q"].shape[:2], device=dev)
    mb = d["table"].shape[1]
    ws = torch.empty(m.msa_attention_workspace(3, 3, 16, 2, mb), dtype=torch.uint8, device=dev)

    def step():
        m.msa_attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["kv"], "BBND", 3, None, out,
                        mb, lse=lse, workspace=ws, softcap=20.0, slopes=d["slopes"],
                        visible=d["visible"])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        c["visible"] = spans(c, "any", i)
        c["slopes"] = c["slopes"] * 0.7
        c["kv"] = torch.tensor([2500 - 600 * i, 300, 77 - i], dtype=torch.int32)
        for n in ("visible", "slopes", "kv"):
            d[n].copy_(c[n])
        graph.replay()
        torch.cuda.synchronize()
        check(c, out.cpu(), lse.cpu())


def test_refusals(dev):
    import block_max_qk_amd as m
    c = make([4], [40], 8, 2, cap=20.0, bias=True, mask="any")
    for kw in (dict(slopes=c["slopes"].double()), dict(slopes=c["slopes"][:4]),
               dict(visible=c["visible"].long()), dict(visible=c["visible"][:3]),
               dict(visible=c["visible"].t().contiguous().t())):
        with pytest.raises(ValueError):
            call({**c, **kw}, dev)
    for cap in (-1.0, float("nan"), float("inf"), 1e-44):
        with pytest.raises(m.MsaError):
            call({**c, "cap": cap}, dev)
    with pytest.raises(ValueError):
        d = {n: (x.to(dev) if torch.is_tensor(x) else x) for n, x in c.items()}
        m.attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["kv"], "BBND",
                    slopes=c["slopes"])


@pytest.mark.parametrize("form", [dict(cap=20.0), dict(bias=True), dict(cap=9.0, bias=True), {}])
def test_ranges_far_into_long_contexts(form, dev):
    """Windows that begin and end past the first 64 blocks, and such that span more
    than 64; each tile's walk and the parts of one."""
    for q_lens, kv_lens in (([1, 1], [20011, 9000]), ([40], [20011]), ([130, 3], [12000, 20011])):
        c = make(q_lens, kv_lens, 4, 1, seed=3, **form)
        pos = pos_of(c)
        for first, end in ((pos - 700, pos - 100), (pos * 0 + 8300, pos * 0 + 8400),
                           (pos * 0 + 130, pos + 1), (pos - 1, pos + 1)):
            c["visible"] = torch.stack([first, end], 1).int()
            log("far", form, q_lens, int(first[0]))
            run(c, dev)


@pytest.mark.parametrize("B", [70, 300])
def test_many_requests(B, dev):
    """Past the 64 requests that one look at the batch holds."""
    gen = torch.Generator().manual_seed(B)
    q = torch.randint(0, 4, (B,), generator=gen).tolist()
    kv = [n + int(x) for n, x in zip(q, torch.randint(0, 500, (B,), generator=gen))]
    kv[7] += 3000
    for form in (dict(cap=20.0, mask="any"), dict(bias=True, mask="documents"), dict(cap=9.0)):
        run(make(q, kv, 8, 2, "BNBD", FP, seed=B, **form), dev)
    q[5] = 200
    kv[5] += 200
    run(make([3 * n for n in q], [n + 600 for n in kv], 8, 2, seed=B, bias=True, mask="any"), dev)
    run(make(q, kv, 8, 2, "TND", BF, seed=B, cap=9.0, mask="any"), dev)


@pytest.mark.parametrize("layout", ["BBND", "BNBD"])
def test_caches_past_4_gib(layout, dev):
    """Pages that begin past 2^32 bytes give the bits that the same ones in a small
    cache do."""
    import block_max_qk_amd as m
    NP, far = 40, (1 << 32) // (128 * 2 * 128 * 2) + 1000
    gen = torch.Generator().manual_seed(9)
    shape = (128, 2, 128) if layout == "BBND" else (2, 128, 128)
    small = [torch.randn(NP, *shape, generator=gen).to(BF).to(dev) for _ in range(2)]
    big = [torch.empty(far + NP, *shape, dtype=BF, device=dev) for _ in range(2)]
    for x, y in zip(big, small):
        x[far:] = y
    for q_lens, kv_lens in (([1, 2], [700, 1500]), ([300], [2000]), ([1500], [2000])):
        T = sum(q_lens)
        q = torch.randn(T, 8, 128, generator=gen).to(BF).to(dev)
        cu = torch.tensor([0, *q_lens]).cumsum(0).int().to(dev)
        kv = torch.tensor(kv_lens).int().to(dev)
        table = torch.randperm(NP, generator=gen)[:len(q_lens) * 16].int().view(-1, 16).to(dev)
        first = torch.randint(0, 600, (T,), generator=gen)
        kw = dict(softcap=20.0, visible=torch.stack([first, first + 900], 1).int().to(dev))
        for form in (kw, {**kw, "softcap": None}, dict(slopes=torch.full((8,), 0.01, device=dev))):
            a = m.attention(q, *small, table, cu, kv, layout, return_lse=True, **form)
            b = m.attention(q, *big, table + far, cu, kv, layout, return_lse=True, **form)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_at_once(dev):
    """Calls of two forms on one cache, from two streams."""
    import block_max_qk_amd as m
    a = make([60, 1], [3000, 400], 8, 2, cap=20.0, mask="documents")
    b = {**a, "cap": 0.0, "slopes": torch.linspace(0, 0.5, 8), "visible": spans(a, "any", 4)}
    want = [call(x, dev) for x in (a, b)]
    d = {n: (x.to(dev) if torch.is_tensor(x) else x) for n, x in a.items()}
    kws = [dict(softcap=20.0, visible=a["visible"].to(dev)),
           dict(slopes=b["slopes"].to(dev), visible=b["visible"].to(dev))]
    streams = [torch.cuda.Stream(dev) for _ in kws]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream(dev))
    got = []
    for _ in range(8):
        got = [m.attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["kv"], "BBND",
                           return_lse=True, stream=s, **kw) for s, kw in zip(streams, kws)]
    torch.cuda.synchronize()
    for (o, lse), (wo, wl) in zip(got, want):
        assert torch.equal(o.cpu(), wo) and torch.equal(lse.cpu(), wl)
