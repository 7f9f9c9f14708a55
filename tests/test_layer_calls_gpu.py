"""Calls of the cache append and the attention that their documentation allows,
each a little off the beaten path: selected blocks without a causal mask, with
missing pages and padded batches, hints and layouts in every form that is
taken, thousands of requests, destinations with other axis orders."""
import sys

import pytest
import torch

import layer_cases as lc
from oracle import layer
from test_append_gpu import angles, batch, bits, make_item
from test_append_gpu import run as run_append
from test_attention_gpu import call, check, reference, to

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


def check_some(c, out, lse, tokens):
    """Some tokens of a case against the oracle, in the case's own mode."""
    keep = torch.tensor(sorted(tokens))
    out, lse = out.cpu(), lse.cpu()
    where = {t: (b, pos) for t, b, pos in layer.positions(c["cu"], c["kv"], c["q"].shape[0])}
    for t in keep.tolist():
        b, pos = where[t]
        first = int(c["kv"][:b].clamp(min=0).sum())
        n = max(pos + 1 if c["mode"] == 3 else int(c["kv"][b]), 0)
        one = dict(c, q=c["q"][t:t + 1], cu=torch.tensor([0, 1], dtype=torch.int32),
                   kv=torch.tensor([n], dtype=torch.int32))
        if c["layout"] == "TND":
            one["k"], one["v"] = (c[x][first:first + n] for x in "kv")
        else:
            one["table"] = c["table"][b:b + 1]
        if c["blocks"] is not None:
            one["blocks"] = c["blocks"][t:t + 1]
        check(one, out[t:t + 1], lse[t:t + 1])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("layout", ["BBND", "BNBD", "TND"])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv", [([1, 5, 0, 2], [900, 400, 300, 1], 8, 2),
                                                   ([400, 1, 300], [1500, 700, 300], 8, 2)])
def test_selected_without_a_causal_mask(layout, dtype, q_lens, kv_lens, Hq, Hkv, dev):
    log("selected, mode 0", layout, dtype, q_lens)
    c = lc.attention_case(q_lens, kv_lens, Hq, Hkv, layout, dtype, mode=0, k=5, seed=130)
    out, lse = call(to(c, dev))
    torch.cuda.synchronize()
    T = sum(q_lens)
    check_some(c, out, lse, {0, 1, 2, T // 2, T - 2, T - 1})


@pytest.mark.parametrize("q_lens,kv_lens", [([2, 1, 4], [700, 500, 3]), ([500, 1, 300], [900, 500, 200])])
def test_selected_with_missing_pages_in_a_padded_batch(q_lens, kv_lens, dev):
    """Pages outside the cache hide their keys; rows that no request holds stay;
    tokens before position 0 and without selected blocks see nothing."""
    c = lc.attention_case(q_lens, kv_lens, 8, 2, k=4, T_extra=19, first=3, width=9, seed=131)
    c["table"][0, 1], c["table"][0, 3], c["table"][1, 0] = -1, c["k"].shape[0], 2 ** 31 - 1
    c["blocks"][4] = -1
    d = to(c, dev)
    T = c["q"].shape[0]
    out = torch.full((T, 8, 128), 3.0, dtype=BF, device=dev)
    lse = torch.full((T, 8), 4.0, device=dev)
    call(d, out, lse)
    torch.cuda.synchronize()
    end = int(c["cu"][-1])
    for rows in (slice(0, 3), slice(end, T)):
        assert (out[rows] == 3).all() and (lse[rows] == 4).all()
    assert (out[4] == 0).all() and (lse[4] == -torch.inf).all()
    check_some(c, out, lse, {3, 4, 5, 3 + q_lens[0] - 1, 3 + q_lens[0], end - 2, end - 1})


@pytest.mark.parametrize("q_lens", [[1, 2], [400, 300]])
def test_selected_lengths_past_the_table_and_one_head_caches(q_lens, dev):
    c = lc.attention_case(q_lens, [512, 512], 6, 1, k=4, seed=132)
    c["kv"] = torch.tensor([2000, 513], dtype=torch.int32)       # the table holds 4 blocks
    c["k"], c["v"] = c["k"][:, :, 0], c["v"][:, :, 0]
    out, lse = call(to(c, dev))
    torch.cuda.synchronize()
    T = sum(q_lens)
    check_some(c, out, lse, {0, q_lens[0], T - 1})


@pytest.mark.parametrize("q_lens,kv,k", [([1, 1], [3000, 40], 0), ([90], [900], 0), ([1, 3], [3000, 40], 5),
                                         ([700], [2000], 5)])
def test_the_forms_of_arguments(q_lens, kv, k, dev):
    """Layouts by name and number, no lse, a table of more rows than requests,
    raw stream handles, queries in wider rows: the same bits."""
    import block_max_qk_amd as m
    c = lc.attention_case(q_lens, kv, 8, 2, k=k, seed=133)
    d = to(c, dev)
    out, lse = call(d)
    mb = d["table"].shape[1]

    def go(layout="BBND", table=d["table"], lse=None, q=d["q"], **kw):
        o = torch.full(c["q"].shape, float("nan"), dtype=BF, device=dev)
        args = (table, d["cu"], d["kv"], layout, 3, None, o, mb)
        if k:
            m.msa_block_attention(q, d["k"], d["v"], d["blocks"], *args, lse=lse, **kw)
        else:
            m.msa_attention(q, d["k"], d["v"], *args, lse=lse, **kw)
        torch.cuda.synchronize()
        assert torch.equal(o, out)

    go()
    go(layout="bbnd")
    go(layout=1)
    go(table=torch.cat([d["table"], torch.full((5, mb), 2 ** 31 - 1, dtype=torch.int32, device=dev)]))
    go(stream=0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    go(stream=s)
    go(stream=s.cuda_stream)
    wide = torch.zeros(c["q"].shape[0], 3, 8, 128, dtype=BF, device=dev)
    wide[:, 1] = d["q"]
    go(q=wide[:, 1])
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
        go()
    if k:
        assert torch.equal(m.block_attention(d["q"], d["k"], d["v"], d["blocks"], d["table"], d["cu"],
                                             d["kv"], "BBND"), out)
    else:
        assert torch.equal(m.attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["kv"], "BBND"),
                           out)
    torch.cuda.synchronize()


@pytest.mark.parametrize("q_lens,kv,k", [([1, 1, 1], [3000, 40, 1], 0), ([60, 1], [2500, 700], 0),
                                         ([300, 500], [2000, 500], 6), ([1, 2], [2000, 300], 6)])
def test_packed_hints(q_lens, kv, k, dev):
    """max_blocks only steers the split of packed keys: 0, too small, too large."""
    import block_max_qk_amd as m
    c = lc.attention_case(q_lens, kv, 8, 2, "TND", FP, k=k, seed=134)
    d = to(c, dev)
    ref = None
    T = sum(q_lens)
    for hint in (0, 1, 5, 24, 1 << 12, 1 << 24):
        out = torch.full(c["q"].shape, float("nan"), dtype=FP, device=dev)
        lse = torch.full((T, 8), float("nan"), device=dev)
        args = (None, d["cu"], d["kv"], "TND", 3, None, out, hint)
        if k:
            m.msa_block_attention(d["q"], d["k"], d["v"], d["blocks"], *args, lse=lse)
        else:
            m.msa_attention(d["q"], d["k"], d["v"], *args, lse=lse)
        torch.cuda.synchronize()
        if T < 100:
            ref = reference(c) if ref is None else ref
            check(c, out, lse, ref)
        else:
            assert torch.isfinite(out).all()
            check_some(c, out, lse, {0, 299, 300, T - 1})


@pytest.mark.parametrize("k", [0, 3])
def test_thousands_of_requests(k, dev):
    """Most of them empty, some without new tokens, in both layouts."""
    gen = torch.Generator().manual_seed(135)
    B = 5000
    q = (torch.rand(B, generator=gen) < 0.05).int() * torch.randint(1, 4, (B,), generator=gen).int()
    kv = torch.where(torch.rand(B, generator=gen) < 0.3, torch.randint(1, 200, (B,), generator=gen), q)
    for layout in ("BBND", "TND"):
        c = lc.attention_case(q.tolist(), kv.tolist(), 2, 1, layout, k=k, seed=136)
        out, lse = call(to(c, dev))
        torch.cuda.synchronize()
        T = c["q"].shape[0]
        check_some(c, out, lse, set(torch.randint(0, T, (40,), generator=gen).tolist()) | {0, T - 1})


def test_append_for_thousands_of_requests(dev):
    gen = torch.Generator().manual_seed(137)
    B = 5000
    q = (torch.rand(B, generator=gen) < 0.05).int() * torch.randint(1, 4, (B,), generator=gen).int()
    kv = torch.where(torch.rand(B, generator=gen) < 0.1, torch.randint(3, 200, (B,), generator=gen), q)
    gen, cu, T, kv, table, pages = batch(q.tolist(), kv.tolist(), 138)
    cos, sin = angles(200, 32)
    for layout in ("BNBD", "TND"):
        src = torch.randn(T, 1, 128, generator=gen).to(BF)
        run_append([make_item(src, kind, layout, T, 1, pages, int(kv.sum()), gen, kind != "same")
                    for kind in ("same", "mxfp4")], cos, sin, table, cu, kv, dev)


def test_append_of_broadcast_rows_and_to_other_axis_orders(dev):
    """Sources with strides of 0; rows whose heads lie outside their tokens."""
    import block_max_qk_amd as m
    gen, cu, T, kv, table, pages = batch([5, 1, 3], [140, 1, 3], 139)
    args = (None, None, table.to(dev), cu.to(dev), kv.to(dev))
    one = torch.randn(1, 1, 128, generator=gen).to(FP).to(dev)
    rows = torch.zeros(4, T, 128, dtype=FP, device=dev)
    cache = torch.zeros(pages, 4, 128, 128, dtype=FP, device=dev)
    codes = torch.zeros(4, T, 64, dtype=torch.uint8, device=dev)
    scale = torch.zeros(T, 4, 4, dtype=torch.uint8, device=dev)
    plain = torch.zeros(T, 4, 64, dtype=torch.uint8, device=dev)
    plain_scale = torch.zeros_like(scale)
    src = one.expand(T, 4, 128)
    heads = torch.randn(T, 1, 128, generator=gen).to(FP).to(dev).expand(T, 4, 128)
    m.msa_cache_append([m.CacheItem(src, rows.transpose(0, 1), "ROWS"),
                        m.CacheItem(heads, cache, "BNBD"),
                        m.CacheItem(heads, codes.transpose(0, 1), "ROWS", scale),
                        m.CacheItem(heads.contiguous(), plain, "rows", plain_scale)], *args)
    torch.cuda.synchronize()
    assert torch.equal(bits(rows), bits(one.expand(4, T, 128)))
    assert torch.equal(codes.transpose(0, 1), plain) and torch.equal(scale, plain_scale)
    for t, b, pos in layer.positions(cu, kv, T):
        assert torch.equal(cache[int(table[b, pos // 128]), :, pos % 128], heads[t])


def test_append_of_one_row_and_of_many_heads(dev):
    gen, cu, T, kv, table, pages = batch([1], [1], 140)
    cos, sin = angles(4, 16)
    for H in (1, 3, 129):
        src = torch.randn(T, H, 128, generator=gen).to(FP)
        for layout in ("BBND", "BNBD", "TND", "ROWS"):
            run_append([make_item(src, kind, layout, T, H, pages, 1, gen, True)
                        for kind in ("same", "e4m3", "e5m2", "i8", "mxfp4")], cos, sin, table, cu, kv,
                       dev, True)


def test_two_calls_at_once_into_one_cache(dev):
    """Two streams append different requests' tokens to one cache, and attend."""
    import block_max_qk_amd as m
    gen = torch.Generator().manual_seed(141)
    table, pages = lc.table_for([300, 200], gen)
    k = torch.zeros(pages, 128, 2, 128, dtype=BF, device=dev)
    v = torch.zeros_like(k)
    cos, sin = (x.to(dev) for x in angles(300, 128))
    rows = [torch.randn(n, 12, 128, generator=gen).to(BF).to(dev) for n in (300, 200)]
    tables = [table[b:b + 1].contiguous().to(dev) for b in (0, 1)]
    streams = [torch.cuda.Stream() for _ in rows]
    torch.cuda.synchronize()
    outs = []
    for x, t, s in zip(rows, tables, streams):
        with torch.cuda.stream(s):
            n = x.shape[0]
            cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
            kv = torch.tensor([n], dtype=torch.int32, device=dev)
            q = torch.empty(n, 8, 128, dtype=BF, device=dev)
            m.msa_cache_append([m.CacheItem(x[:, :8], q, "ROWS", rotate=True),
                                m.CacheItem(x[:, 8:10], k, "BBND", rotate=True),
                                m.CacheItem(x[:, 10:], v, "BBND")], cos, sin, t, cu, kv)
            outs.append((q, *m.attention(q, k, v, t, cu, kv, "BBND", return_lse=True)))
    torch.cuda.synchronize()
    for (q, out, lse), t, n in zip(outs, tables, (300, 200)):
        c = {"q": q.cpu(), "k": k.cpu(), "v": v.cpu(), "table": t.cpu(), "layout": "BBND", "mode": 3,
             "cu": torch.tensor([0, n], dtype=torch.int32), "kv": torch.tensor([n], dtype=torch.int32),
             "blocks": None}
        check_some(c, out, lse, {0, 1, 127, 128, n - 1})


@pytest.mark.parametrize("q_lens", [[1], [3], [700]])
def test_the_longest_lengths(q_lens, dev):
    """2^31 - 1 keys behind a table of 2^24 blocks: the last blocks' selection
    gives the bits of a short request's, and the append finds the last slots."""
    import block_max_qk_amd as m
    T, near, MB = sum(q_lens), 8, 1 << 24
    c = lc.attention_case(q_lens, [near * 128 - 1], 8, 1, k=3, seed=142)
    d = to(c, dev)
    want = call(d)
    far = dict(d)
    far["table"] = torch.full((1, MB), -1, dtype=torch.int32, device=dev)
    far["table"][0, MB - near:] = d["table"][0]
    far["kv"] = torch.tensor([2 ** 31 - 1], dtype=torch.int32, device=dev)
    far["blocks"] = torch.where(d["blocks"] >= 0, d["blocks"] + (MB - near), d["blocks"])
    got = call(far)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    gen = torch.Generator().manual_seed(143)
    src = torch.randn(T, 1, 128, generator=gen).to(BF).to(dev)
    for x in (d, far):
        x["cache"] = torch.zeros_like(d["k"])
        m.msa_cache_append([m.CacheItem(src, x["cache"], "BBND")], None, None, x["table"], x["cu"],
                           x["kv"])
    torch.cuda.synchronize()
    assert torch.equal(far["cache"], d["cache"])
    assert int((d["cache"] != 0).any(-1).sum()) == T
