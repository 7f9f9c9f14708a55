"""The attention entry points against the binary64 oracle (oracle/layer.py),
within bounds derived from the arithmetic (``attention_bounds`` there), through
each kernel: 16-row tiles, 128- and 256-row tiles, with and without a split
over the keys, and the selected blocks' form."""
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


def to(c, dev):
    return {n: (x.to(dev) if torch.is_tensor(x) else x) for n, x in c.items()}


def call(d, out=None, lse=None, **kw):
    """(out, lse) of the case; outputs start as NaN, so that a row that is not
    written shows."""
    import block_max_qk_amd as m
    q = d["q"]
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=q.device) if out is None else out
    lse = torch.full(q.shape[:2], float("nan"), device=q.device) if lse is None else lse
    mb = d["table"].shape[1] if d["table"] is not None else (d["k"].shape[0] + 127) // 128
    args = (d["table"], d["cu"], d["kv"], d["layout"], d["mode"], d.get("scale"), out, mb)
    if d["blocks"] is not None:
        m.msa_block_attention(q, d["k"], d["v"], d["blocks"], *args, lse=lse, **kw)
    else:
        m.msa_attention(q, d["k"], d["v"], *args, lse=lse, **kw)
    return out, lse


def reference(c):
    return layer.attention(c["q"], c["k"], c["v"], c["table"], c["cu"], c["kv"], c["layout"],
                           c["mode"], c.get("scale"), c["blocks"])


def check(c, out, lse, ref=None):
    ref = reference(c) if ref is None else ref
    first, end = int(c["cu"][0]), int(c["cu"][-1])
    out, lse = out.cpu().double()[first:end], lse.cpu().double()[first:end]
    tol_out, tol_lse = layer.attention_bounds(ref, c["q"].dtype)
    ref = layer.Attention(*(x[first:end] for x in ref))
    assert torch.isfinite(out).all()
    worst = ((out - ref.out).abs() / tol_out[first:end].clamp(min=1e-30)).max()
    assert ((out - ref.out).abs() <= tol_out[first:end]).all(), float(worst)
    empty = ref.keys == 0
    assert (out[empty] == 0).all()
    assert torch.equal(lse == -torch.inf, empty)
    d = (lse - ref.lse).abs()[~empty]
    assert (d <= tol_lse[first:end][~empty]).all(), float(d.max())
    return float(worst)


def run(c, dev):
    out, lse = call(to(c, dev))
    torch.cuda.synchronize()
    return check(c, out, lse)


# every layout and type, group sizes from one head to more than a tile
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("layout", ["BBND", "BNBD", "TND"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (10, 2), (16, 1), (12, 4), (40, 2)])
def test_decode(dtype, layout, Hq, Hkv, dev):
    log("decode", dtype, layout, Hq, Hkv)
    run(lc.attention_case([1, 1, 0, 1, 1], [1, 127, 300, 128, 577], Hq, Hkv, layout, dtype,
                          seed=Hq), dev)


@pytest.mark.parametrize("layout", ["BBND", "BNBD", "TND"])
@pytest.mark.parametrize("mode", [0, 3])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv", [
    ([33], [33], 8, 2), ([1, 2, 3], [200, 2, 131], 8, 1), ([70, 1, 9], [70, 300, 129], 6, 2),
    ([129], [260], 4, 4), ([17, 40], [65, 64 + 40], 24, 1), ([5], [700], 300, 1),
])
def test_chunks(layout, mode, q_lens, kv_lens, Hq, Hkv, dev):
    log("chunks", layout, mode, q_lens, Hq, Hkv)
    run(lc.attention_case(q_lens, kv_lens, Hq, Hkv, layout, BF if Hq % 4 else FP, mode,
                          seed=sum(q_lens)), dev)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_many_rows_and_tiles(dtype, dev):
    """Enough rows for 256-row tiles, ragged ends of tiles and stages."""
    log("256-row tiles", dtype)
    run(lc.attention_case([515, 301], [515, 430], 64, 8, "BBND", dtype, seed=5), dev)


def test_split_over_keys(dev):
    import block_max_qk_amd as m
    for q_lens, kv_lens, Hq, Hkv in (([1, 1], [5000, 129], 16, 2), ([40], [3333], 16, 2)):
        c = lc.attention_case(q_lens, kv_lens, Hq, Hkv, seed=len(q_lens))
        assert m.msa_attention_workspace(sum(q_lens), len(q_lens), Hq, Hkv,
                                         c["table"].shape[1]) > 0
        log("split", q_lens, kv_lens)
        run(c, dev)


def test_one_token_everything(dev):
    run(lc.attention_case([1], [1], 1, 1, "TND"), dev)
    run(lc.attention_case([1], [1], 1, 1, "BBND"), dev)


@pytest.mark.parametrize("layout", ["BBND", "TND"])
def test_rows_that_see_nothing(layout, dev):
    """Empty requests, tokens before position 0, no keys at all: out 0, lse -inf."""
    run(lc.attention_case([3, 0, 5, 4], [0, 77, 2, 300], 8, 2, layout, seed=7), dev)
    run(lc.attention_case([50, 200], [20, 0], 8, 2, layout, seed=8), dev)
    run(lc.attention_case([4, 2], [0, 0], 8, 2, layout, mode=0, seed=9), dev)


def test_padded_batch_rows_stay(dev):
    """Rows behind the last request and before the first keep what they held."""
    for q_lens, kv in (([2, 1], [400, 30]), ([60, 30], [60, 500])):
        c = lc.attention_case(q_lens, kv, 8, 2, T_extra=21, first=5, seed=11)
        d = to(c, dev)
        T = c["q"].shape[0]
        out = torch.full((T, 8, 128), 3.0, dtype=BF, device=dev)
        lse = torch.full((T, 8), 4.0, device=dev)
        call(d, out, lse)
        torch.cuda.synchronize()
        end = int(c["cu"][-1])
        for rows in (slice(0, 5), slice(end, T)):
            assert (out[rows] == 3).all() and (lse[rows] == 4).all()
        check(c, out, lse)


def test_pages_outside_the_cache(dev):
    """Table entries that name no page hide their keys (and are not read)."""
    for q_lens, kv in (([1, 1], [500, 300]), ([70], [700])):
        c = lc.attention_case(q_lens, kv, 8, 2, seed=13, width=8)
        pages = c["k"].shape[0]
        c["table"][0, 1] = -7
        c["table"][0, 2] = pages
        c["table"][-1, 0] = 2 ** 31 - 1
        run(c, dev)


def test_wide_table_and_lengths_past_it(dev):
    c = lc.attention_case([1, 3], [130, 64], 8, 2, seed=14, width=700)
    run(c, dev)
    c = lc.attention_case([1, 90], [256, 256], 8, 2, seed=15)
    c["kv"] = torch.tensor([900, 1000], dtype=torch.int32)     # the table holds 2 blocks
    run(c, dev)
    c = lc.attention_case([2, 3], [100, 40], 8, 2, "TND", seed=16)
    c["kv"] = torch.tensor([100, 400], dtype=torch.int32)      # the tensor holds 140 keys
    run(c, dev)


@pytest.mark.parametrize("layout", ["BBND", "BNBD"])
def test_odd_strides(layout, dev):
    """Queries in wider rows, keys and values as two planes of one cache and
    with gaps between pages."""
    c = lc.attention_case([2, 70], [200, 333], 8, 2, layout, seed=17)
    d = to(c, dev)
    wide = torch.full((c["q"].shape[0], 20, 128), float("nan"), dtype=BF, device=dev)
    wide[:, 3:11] = d["q"]
    d["q"] = wide[:, 3:11]
    both = torch.full((c["k"].shape[0], 3, *c["k"].shape[1:]), float("nan"), dtype=BF, device=dev)
    both[:, 0], both[:, 2] = d["k"], d["v"]
    d["k"], d["v"] = both[:, 0], both[:, 2]
    out, lse = call(d, out=torch.empty(c["q"].shape, dtype=BF, device=dev))
    torch.cuda.synchronize()
    check(c, out, lse)


def test_three_axis_cache(dev):
    c = lc.attention_case([1, 20], [200, 333], 8, 1, "BBND", seed=18)
    c["k"], c["v"] = c["k"][:, :, 0], c["v"][:, :, 0]
    run(c, dev)


def test_packed_rows_of_a_projection(dev):
    c = lc.attention_case([45, 1, 130], [45, 1, 130], 8, 2, "TND", FP, seed=19)
    qkv = torch.cat([c["q"], c["k"], c["v"]], dim=1).to(dev)
    d = to(c, dev)
    d["q"], d["k"], d["v"] = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    out, lse = call(d, out=torch.empty(c["q"].shape, dtype=FP, device=dev))
    torch.cuda.synchronize()
    check(c, out, lse)


@pytest.mark.parametrize("q_lens,kv", [([1, 1], [200, 77]), ([90], [300])])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_keys_behind_the_last(q_lens, kv, bad, dev):
    """What unused slots and pages hold never reaches a result."""
    c = lc.attention_case(q_lens, kv, 8, 2, seed=20)
    ref = reference(c)
    used = torch.zeros(c["k"].shape[0], 128, dtype=torch.bool)
    for b, n in enumerate(kv):
        for i in range(-(-n // 128)):
            used[int(c["table"][b, i]), :max(0, min(128, n - 128 * i))] = True
    for x in (c["k"], c["v"]):
        x[~used] = bad
    out, lse = call(to(c, dev))
    torch.cuda.synchronize()
    check(c, out, lse, ref)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("q_lens,kv,Hq,Hkv,k", [
    ([3], [300], 4, 1, 0), ([5, 1], [40, 9], 6, 3, 0), ([90], [300], 8, 2, 0),
    ([700], [700], 16, 2, 0), ([2, 33], [300, 700], 300, 1, 0), ([40], [3333], 16, 2, 0),
    ([70, 90], [1000, 513], 16, 2, 5), ([2100], [2200], 8, 2, 4)])
def test_nonfinite_values_that_a_row_does_not_see(bad, q_lens, kv, Hq, Hkv, k, dev):
    """The last token's key and value hold no numbers: rows of earlier tokens
    (in the same tile) and of tokens that did not select its block are as they
    would be without."""
    log("unseen", bad, q_lens, Hq, k)
    c = lc.attention_case(q_lens, kv, Hq, Hkv, k=k, seed=22)
    page, slot = int(c["table"][0, (kv[0] - 1) // 128]), (kv[0] - 1) % 128
    n = q_lens[0]
    full = dict(c, k=c["k"].clone(), v=c["v"].clone())
    full["v"][page, slot, :, 3:90] = bad
    full["k"][page, slot, 0, 5] = bad
    out, lse = (x.cpu() for x in call(to(full, dev)))
    torch.cuda.synchronize()
    clean_out, clean_lse = (x.cpu() for x in call(to(c, dev)))
    see = torch.zeros(c["q"].shape[0], Hkv, dtype=torch.bool)
    see[n - 1] = True
    if k:
        see &= (c["blocks"] == (kv[0] - 1) // 128).any(-1)
    rows = see.repeat_interleave(Hq // Hkv, 1)
    assert torch.equal(out[~rows], clean_out[~rows]) and torch.equal(lse[~rows], clean_lse[~rows])
    if rows.any():
        assert not torch.isfinite(out[rows][:, 3:90]).any()


def test_large_and_small_scores(dev):
    """Scores far apart (weights that underflow, a maximum that grows along the
    keys) and a scale of its own."""
    for q_lens, kv in (([1], [900]), ([100], [900])):
        c = lc.attention_case(q_lens, kv, 8, 2, seed=21)
        ramp = torch.linspace(0.05, 4, 128)[None, :, None, None]
        c["k"] = (c["k"].float() * ramp).to(BF)
        c["scale"] = 1.5
        run(c, dev)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("layout", ["BBND", "BNBD", "TND"])
@pytest.mark.parametrize("k,Hq,Hkv", [(1, 8, 1), (4, 16, 4), (16, 12, 4), (64, 40, 2)])
def test_selected(dtype, layout, k, Hq, Hkv, dev):
    log("selected", dtype, layout, k, Hq, Hkv)
    run(lc.attention_case([1, 3, 0, 30], [1, 2000, 55, 999], Hq, Hkv, layout, dtype, k=k,
                          seed=k), dev)


def check_tokens(c, out, lse, tokens):
    """Compare some tokens' rows, each as a request of its own (causal mode)."""
    out, lse = out.cpu(), lse.cpu()
    where = {t: (b, pos) for t, b, pos in layer.positions(c["cu"], c["kv"], c["q"].shape[0])}
    for t in tokens:
        b, pos = where[t]
        first = int(c["kv"][:b].clamp(min=0).sum())
        one = dict(c, q=c["q"][t:t + 1], cu=torch.tensor([0, 1], dtype=torch.int32),
                   kv=torch.tensor([pos + 1], dtype=torch.int32))
        if c["layout"] == "TND":
            one["k"], one["v"] = (c[x][first:first + pos + 1] for x in "kv")
        else:
            one["table"] = c["table"][b:b + 1]
        if c["blocks"] is not None:
            one["blocks"] = c["blocks"][t:t + 1]
        check(one, out[t:t + 1], lse[t:t + 1])


@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (16, 8), (40, 2), (4, 4), (300, 1)])
@pytest.mark.parametrize("layout", ["BBND", "BNBD", "TND"])
def test_selected_long_chunks(layout, Hq, Hkv, dev):
    """Long enough for the tiles that walk the union of their tokens' blocks."""
    log("selected chunks", layout, Hq, Hkv)
    q_lens, kv = ([250, 131], [1000, 131]) if Hkv > 2 else ([900, 1170], [2000, 1170])
    if Hq == 300:
        q_lens, kv = [2050], [2300]
    c = lc.attention_case(q_lens, kv, Hq, Hkv, layout, FP if Hq == 16 else BF, k=5, seed=Hq)
    out, lse = call(to(c, dev))
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    T, gen = sum(q_lens), torch.Generator().manual_seed(Hq)
    some = {0, 1, 5, 6, 7, 31, 32, 255, T - 1, T - 2, q_lens[0] - 1, q_lens[0] % T}
    some |= set(torch.randint(0, T, (20,), generator=gen).tolist())
    check_tokens(c, out, lse, sorted(x for x in some if x < T))


def test_selected_chunk_any_order_and_wide_spans(dev):
    """Lists out of order, with repeats and entries that name nothing, over more
    blocks than a workgroup marks at a time."""
    gen = torch.Generator().manual_seed(33)
    T, Hkv, k, nb = 2100, 2, 9, 5000
    c = lc.attention_case([T], [T + 300], 4, Hkv, k=k, seed=34)
    c["blocks"] = torch.randint(-3, 25, (T, Hkv, k), generator=gen, dtype=torch.int32)
    c["blocks"][::7, :, 2] = 2 ** 31 - 1
    c["blocks"][::5, :, 1] = -2 ** 31
    out, lse = call(to(c, dev))
    torch.cuda.synchronize()
    check_tokens(c, out, lse, range(0, T, 29))
    # 5000 blocks behind few pages
    c = lc.attention_case([T], [T], 4, Hkv, k=k, seed=35)
    last = nb * 128 - 60
    c["table"] = (torch.arange(nb) % c["k"].shape[0]).int()[None]
    c["kv"] = torch.tensor([last], dtype=torch.int32)
    c["blocks"] = torch.randint(0, nb, (T, Hkv, k), generator=gen, dtype=torch.int32)
    c["blocks"][..., 0] = ((last - T + torch.arange(T)) // 128)[:, None]
    out, lse = call(to(c, dev))
    torch.cuda.synchronize()
    check_tokens(c, out, lse, (0, 63, 1000, T - 1))


def test_selected_any_order_and_repeats(dev):
    c = lc.attention_case([1, 5], [1000, 700], 8, 2, k=8, seed=23)
    T = c["q"].shape[0]
    rows = torch.tensor([
        [3, 1, 3, -1, 0, 1, 900, 2], [-1, -1, -1, -1, -1, -1, -1, -1], [5, -1, 5, 4, -9, 4, 5, 5],
        [7, 6, 5, 4, 3, 2, 1, 0], [0, 0, 0, 0, 0, 0, 0, 0], [2 ** 31 - 1, 2, -2 ** 31, 2, 2, 0, 1, 1],
    ], dtype=torch.int32)
    c["blocks"] = torch.stack([rows, rows.flip(1)], dim=1)[:T].contiguous()
    run(c, dev)


def test_selected_all_blocks_is_dense(dev):
    c = lc.attention_case([1, 40], [513, 300], 8, 2, seed=24)
    s = dict(c, blocks=torch.arange(5, dtype=torch.int32).expand(41, 2, 5).contiguous())
    run(s, dev)
    a, b = call(to(c, dev)), call(to(s, dev))
    # both lie within the bounds of one definition
    ref = reference(c)
    tol_out, tol_lse = layer.attention_bounds(ref, BF)
    assert ((a[0] - b[0]).abs().cpu().double() <= 2 * tol_out).all()
    assert ((a[1] - b[1]).abs().cpu().double() <= 2 * tol_lse).all()


def test_large_batch(dev):
    """More requests than one scan of the batch holds."""
    gen = torch.Generator().manual_seed(3)
    q = torch.randint(0, 3, (150,), generator=gen).tolist()
    kv = [n + int(x) for n, x in zip(q, torch.randint(0, 200, (150,), generator=gen))]
    run(lc.attention_case(q, kv, 4, 2, seed=25), dev)
    run(lc.attention_case(q, kv, 4, 2, "TND", seed=26), dev)
    run(lc.attention_case(q, kv, 4, 2, k=2, seed=27), dev)


@pytest.mark.parametrize("layout", ["BBND", "TND"])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,k", [
    ([1] * 9, [9000, 1, 0, 130, 128, 127, 300, 40, 6000], 16, 2, 0),
    ([0, 1, 0, 1], [500, 2049, 0, 1], 8, 1, 0),
    ([5, 1, 7, 2, 0, 3, 1, 1, 1, 1, 1, 1], [4000, 1500, 7, 1, 10, 2600] + [1025] * 6, 8, 2, 0),
    ([1, 1, 1], [3000, 1600, 90], 40, 2, 0),
    ([1] * 64, [5000] + [100 * (i % 13) for i in range(63)], 4, 2, 0),
    ([1, 0] * 65, [64 * (i % 40) for i in range(129)] + [7000], 4, 1, 0),
    ([300, 20, 1, 40], [9000, 20, 3000, 700], 16, 2, 0),
    ([120, 9, 0, 2], [9000, 40, 300, 2], 16, 8, 6),
    ([1, 1, 1, 1], [9000, 40, 0, 2500], 16, 4, 20),
])
def test_uneven_batches(layout, q_lens, kv_lens, Hq, Hkv, k, dev):
    """Long requests in many parts beside whole ones, and requests of none;
    nothing is read of the workspace that the call did not write."""
    import block_max_qk_amd as m
    c = lc.attention_case(q_lens, kv_lens, Hq, Hkv, layout, k=k, seed=80)
    d = to(c, dev)
    mb = d["table"].shape[1] if d["table"] is not None else (d["k"].shape[0] + 127) // 128
    need = m.msa_attention_workspace(d["q"].shape[0], len(q_lens), Hq, Hkv, mb,
                                     0 if d["blocks"] is None else d["blocks"].shape[2])
    got = []
    for fill in (255, 0x41):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device=dev)
        got.append(call(d, workspace=ws[:need]) if need else call(d))
        torch.cuda.synchronize()
        assert (ws[need:] == fill).all()
    check(c, *got[0])
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_same_bits_every_time(dev):
    for c in (lc.attention_case([1, 1], [5000, 129], 16, 2, seed=28),
              lc.attention_case([200], [1000], 16, 2, seed=29),
              lc.attention_case([1, 30], [3000, 900], 16, 2, k=6, seed=30)):
        d = to(c, dev)
        a, b = call(d), call(d)
        torch.cuda.synchronize()
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16))
        assert torch.equal(a[1].view(torch.int32), b[1].view(torch.int32))


def test_allocating_forms(dev):
    import block_max_qk_amd as m
    c = lc.attention_case([1, 1], [5000, 129], 16, 2, k=3, seed=31)
    d = to(c, dev)
    out, lse = m.block_attention(d["q"], d["k"], d["v"], d["blocks"], d["table"], d["cu"], d["kv"],
                                 "BBND", return_lse=True)
    check(c, out, lse)
    c["blocks"] = d["blocks"] = None
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = m.attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["kv"], "BBND",
                           return_lse=True, stream=s)
    s.synchronize()
    check(c, out, lse)
    only = m.attention(d["q"], d["k"], d["v"], d["table"], d["cu"], d["kv"], "BBND")
    assert torch.equal(only, out)
