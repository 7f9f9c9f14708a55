"""The 256-row tiles (long chunks and prompts) against the oracle and, bit for
bit, against the 128-row tiles: every layout and type, whole and split, odd
groups, keys and values that a row does not see; and batches of many decode
tokens beside a long chunk, or of more items than are split.  Each test asserts
the tile that its sizes choose."""
import sys

import pytest
import torch

import layer_cases as lc
import tile_cases
from oracle import layer
from test_attention_gpu import call, check, to
from test_attention_gpu import test_nonfinite_values_that_a_row_does_not_see as unseen

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


def plan(c):
    """(tile rows, workspace bytes) of the case."""
    import block_max_qk_amd as m
    T, Hq, _ = c["q"].shape
    Hkv = c["k"].shape[2 if c["layout"] == "BBND" else 1]
    mb = c["table"].shape[1] if c["table"] is not None else (c["k"].shape[0] + 127) // 128
    at = (T, len(c["kv"]), Hq, Hkv, mb, 0 if c["blocks"] is None else c["blocks"].shape[2])
    return m.msa_attention_tile_rows(*at), m.msa_attention_workspace(*at)


def check_rows(c, out, lse, tokens, heads=None):
    """Some tokens' rows against the oracle, each token a request of its own
    (the heads of some KV heads only, for large groups)."""
    out, lse = out.cpu(), lse.cpu()
    where = {t: (b, pos) for t, b, pos in layer.positions(c["cu"], c["kv"], c["q"].shape[0])}
    for t in tokens:
        b, pos = where[t]
        first = int(c["kv"][:b].clamp(min=0).sum())
        n = pos + 1 if c["mode"] == 3 else int(c["kv"][b])
        one = dict(c, q=c["q"][t:t + 1], cu=torch.tensor([0, 1], dtype=torch.int32),
                   kv=torch.tensor([n], dtype=torch.int32))
        if c["layout"] == "TND":
            one["k"], one["v"] = (c[x][first:first + n] for x in "kv")
        else:
            one["table"] = c["table"][b:b + 1]
        check(one, out[t:t + 1], lse[t:t + 1])


def some_tokens(q_lens, gen, extra=6):
    """The ends of every request and of the tiles about them, and a few others."""
    T, at, picks = sum(q_lens), 0, set()
    for n in q_lens:
        if n:
            picks |= {at, at + n - 1, at + n // 2}
        at += n
    return sorted(picks | set(torch.randint(0, T, (extra,), generator=gen).tolist()))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("name", list(tile_cases.CASES))
def test_rows_against_the_oracle(name, dtype, dev):
    log("256 rows", name, dtype)
    q_lens, kv_lens, Hq, Hkv, layout, width, split = tile_cases.CASES[name]
    c = lc.attention_case(q_lens, kv_lens, Hq, Hkv, layout, dtype, width=width, seed=110)
    rows, need = plan(c)
    assert rows == 256 and (need > 0) == split
    out, lse = call(to(c, dev))
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    check_rows(c, out, lse, some_tokens(q_lens, torch.Generator().manual_seed(111)))


@pytest.mark.parametrize("q_lens,kv_lens", [([1000], [1000]), ([301, 0, 700, 33], [301, 9, 830, 700])])
@pytest.mark.parametrize("layout", ["BBND", "TND"])
def test_without_a_causal_mask(q_lens, kv_lens, layout, dev):
    width = 16 if layout == "BBND" else None
    c = lc.attention_case(q_lens, kv_lens, 64, 8, layout, BF, mode=0, seed=112, width=width)
    assert plan(c)[0] == 256
    out, lse = call(to(c, dev))
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    check_rows(c, out, lse, some_tokens(q_lens, torch.Generator().manual_seed(113)))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("layout", ["BBND", "BNBD", "TND"])
@pytest.mark.parametrize("Hq,Hkv,T", [(64, 8, 1000), (40, 8, 1640)])
def test_every_row_is_the_128_row_tiles(layout, dtype, Hq, Hkv, T, dev):
    """A whole tile's rows have the bits that 128-row tiles give them, called
    with a few tokens at a time (a row's bits do not depend on its tile)."""
    c = lc.attention_case([T], [T], Hq, Hkv, layout, dtype, seed=114)
    log("bits", layout, dtype, Hq, T)
    assert plan(c) == (256, 0)
    out, lse = call(to(c, dev))
    step = 48
    for t in range(0, T, step):
        n = min(step, T - t)
        e = t + n
        part = dict(c, q=c["q"][t:e], cu=torch.tensor([0, n], dtype=torch.int32),
                    kv=torch.tensor([e], dtype=torch.int32))
        if layout == "TND":
            part["k"], part["v"] = c["k"][:e], c["v"][:e]
        else:
            part["table"] = c["table"][:, :-(-e // 128)].contiguous()
        if e > 1024:             # (such a part is split over the keys)
            break
        assert plan(part) == (128, 0)
        po, pl = call(to(part, dev))
        assert torch.equal(po, out[t:e]) and torch.equal(pl, lse[t:e]), t


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("q_lens,kv,Hq,Hkv", [
    ([1000], [1000], 64, 8), ([520], [6000], 64, 8), ([330, 600], [9000, 2000], 64, 8),
    ([70], [2048], 600, 2)])
def test_values_that_a_row_does_not_see(bad, q_lens, kv, Hq, Hkv, dev):
    assert plan(lc.attention_case(q_lens, kv, Hq, Hkv, seed=22))[0] == 256
    unseen(bad, q_lens, kv, Hq, Hkv, 0, dev)


def test_rows_that_see_nothing_and_rows_that_no_request_holds(dev):
    """Tokens before position 0, an empty request's tokens, rows behind the last
    request and before the first; pages that are not there."""
    q_lens, kv_lens = [600, 300, 200], [700, 0, 100]
    c = lc.attention_case(q_lens, kv_lens, 64, 8, "BBND", BF, T_extra=77, first=9, width=16, seed=115)
    c["table"][0, 1], c["table"][0, 2] = -5, c["k"].shape[0]
    assert plan(c)[0] == 256
    d = to(c, dev)
    T = c["q"].shape[0]
    out = torch.full((T, 64, 128), 3.0, dtype=BF, device=dev)
    lse = torch.full((T, 64), 4.0, device=dev)
    call(d, out, lse)
    torch.cuda.synchronize()
    end = int(c["cu"][-1])
    for rows in (slice(0, 9), slice(end, T)):
        assert (out[rows] == 3).all() and (lse[rows] == 4).all()
    none = [slice(9 + 600, 9 + 900), slice(9 + 900, 9 + 1000)]      # no keys; before position 0
    for rows in none:
        assert (out[rows] == 0).all() and (lse[rows] == -torch.inf).all()
    for t in (9, 9 + 300, 9 + 599, 9 + 1000, end - 1):
        b = 0 if t < 609 else 2
        pos = int(c["kv"][b]) - (q_lens[b]) + t - int(c["cu"][b])
        one = dict(c, q=c["q"][t:t + 1], cu=torch.tensor([0, 1], dtype=torch.int32),
                   kv=torch.tensor([pos + 1], dtype=torch.int32), table=c["table"][b:b + 1])
        check(one, out[t:t + 1].cpu(), lse[t:t + 1].cpu())


def test_odd_strides(dev):
    """Queries in wider rows, keys and values as planes of one cache."""
    q_lens, kv_lens = [700, 300], [2000, 333]
    for layout in ("BBND", "BNBD"):
        c = lc.attention_case(q_lens, kv_lens, 64, 8, layout, FP, seed=116)
        assert plan(c)[0] == 256
        d = to(c, dev)
        plain = call(d)
        wide = torch.full((1000, 70, 128), float("nan"), dtype=FP, device=dev)
        wide[:, 3:67] = d["q"]
        both = torch.full((c["k"].shape[0], 3, *c["k"].shape[1:]), float("nan"), dtype=FP, device=dev)
        both[:, 0], both[:, 2] = d["k"], d["v"]
        d["q"], d["k"], d["v"] = wide[:, 3:67], both[:, 0], both[:, 2]
        out, lse = call(d, out=torch.empty(1000, 64, 128, dtype=FP, device=dev),
                        lse=torch.empty(1000, 64, device=dev))
        torch.cuda.synchronize()
        assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])


def test_graph_replays(dev):
    """Captured with its workspace and replayed, with eager work between."""
    for name in ("one prompt, whole", "parts of both requests"):
        q_lens, kv_lens, Hq, Hkv, layout, width, _ = tile_cases.CASES[name]
        c = lc.attention_case(q_lens, kv_lens, Hq, Hkv, layout, BF, width=width, seed=117)
        d = to(c, dev)
        eager = call(d)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out, lse = call(d)
        torch.cuda.current_stream().wait_stream(s)
        for _ in range(3):
            out.fill_(7.0)
            lse.fill_(7.0)
            call(d)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv", [
    ([1] * 63 + [200], [50 * (i % 9) + 1 for i in range(63)] + [8000], 8, 8),
    ([1] * 63 + [65], [50 * (i % 9) + 1 for i in range(63)] + [8000], 16, 2),
    ([900] + [1] * 63, [2000] + [300] * 63, 4, 4),
])
def test_many_decode_tokens_beside_a_chunk(q_lens, kv_lens, Hq, Hkv, dev):
    """Decode tokens and a chunk of many 16-row tiles in one launch."""
    c = lc.attention_case(q_lens, kv_lens, Hq, Hkv, seed=118)
    assert plan(c)[0] == 16
    out, lse = call(to(c, dev))
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    T = sum(q_lens)
    check_rows(c, out, lse, sorted({0, 1, 40, 62, 63, 64, 100, T - 2, T - 1}))


@pytest.mark.parametrize("layout", ["BBND", "TND"])
def test_large_uneven_decode_batch(layout, dev):
    """1024 items: tiles that are not split, one far longer than the rest."""
    kv_lens = [64 * (i % 17) for i in range(127)] + [20000]
    c = lc.attention_case([1] * 128, kv_lens, 16, 8, layout, seed=119)
    assert plan(c) == (16, 0)
    out, lse = call(to(c, dev))
    torch.cuda.synchronize()
    check_rows(c, out, lse, [0, 1, 16, 63, 64, 100, 126, 127])
