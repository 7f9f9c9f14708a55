"""float16 attention of rows whose largest score lies far above the others (a
sink): the many keys below it keep their share of the result, through each
kernel, whole and split over the keys.

The first key scores `gap` nats above all the others, whose weights are about
e^-gap of its own; with tens of thousands of them their sum is a visible share
of the softmax, and as the sink's value is almost nothing, it is the result."""
import math
import sys

import pytest
import torch

import layer_cases as lc
from test_attention_gpu import call, check_tokens, to

pytestmark = pytest.mark.gpu

FP = torch.float16
AXIS = 24.0              # the queries' part along the sink's key


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_max_qk_amd
    block_max_qk_amd.load_library()
    return torch.device("cuda:0")


def sink_case(q_lens, kv_lens, Hq, Hkv, layout, gap, sink_at=0, **kw):
    """Scores of `gap` at key `sink_at` of every request and of 0 with a spread
    of a quarter elsewhere; values about 1, the sink's about 2^-10."""
    c = lc.attention_case(q_lens, kv_lens, Hq, Hkv, layout, FP, **kw)
    c["q"] *= 0.25
    c["q"][..., 0] = AXIS
    c["k"][..., 0] = 0
    c["v"] = (1 + 0.125 * c["v"].float()).to(FP)
    first = 0
    for b, n in enumerate(kv_lens):
        if n > sink_at:
            if layout == "TND":
                at = (first + sink_at,)
            else:
                page, slot = int(c["table"][b, sink_at // 128]), sink_at % 128
                at = (page, slot) if layout == "BBND" else (page, slice(None), slot)
            c["k"][at] = 0
            c["k"][at][..., 0] = gap * math.sqrt(128) / AXIS
            c["v"][at] = c["v"][at] * 2.0 ** -10
        first += n
    return c


def run(c, dev, tokens):
    out, lse = call(to(c, dev))
    torch.cuda.synchronize()
    check_tokens(c, out, lse, tokens)


@pytest.mark.parametrize("gap", [12.0, 17.0, 18.0, 20.0])
@pytest.mark.parametrize("layout", ["BBND", "BNBD", "TND"])
def test_decode(gap, layout, dev):
    """16-row tiles, split over the keys."""
    log("sink decode", gap, layout)
    run(sink_case([1, 1], [32768, 5000], 8, 2, layout, gap, seed=100), dev, (0, 1))


@pytest.mark.parametrize("gap", [17.0, 20.0])
def test_decode_whole(gap, dev):
    """16-row tiles, not split: as many tiles as the chip takes at once."""
    log("sink whole", gap)
    run(sink_case([1] * 128, [8192] + [140] * 127, 16, 8, "BBND", gap, seed=101), dev, (0, 5))


@pytest.mark.parametrize("gap", [12.0, 18.0])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv", [
    ([40], [32768], 8, 2),           # 128-row tiles, split evenly
    ([100, 60], [20000, 900], 8, 2),   # split by length
    ([20] * 130, [16384] + [30] * 129, 32, 8),   # whole
    ([4096], [32768], 8, 8),         # 256-row tiles, split evenly
    ([8192], [32768], 8, 8),         # whole
])
def test_chunks(gap, q_lens, kv_lens, Hq, Hkv, dev):
    log("sink chunk", gap, q_lens[:3])
    T = sum(q_lens)
    run(sink_case(q_lens, kv_lens, Hq, Hkv, "BBND", gap, seed=102), dev,
        sorted({0, q_lens[0] - 1, T // 2, T - 1}))


@pytest.mark.parametrize("gap", [8.0, 18.0])
@pytest.mark.parametrize("q_lens,kv_lens,Hkv", [([1, 1], [9000, 700], 2), ([3, 9], [9000, 900], 1),
                                                ([900], [8192], 2)])
def test_selected(gap, q_lens, kv_lens, Hkv, dev):
    """Selected blocks, the sink's among them: one token a workgroup, and the
    union of a long chunk's lists."""
    log("sink selected", gap, q_lens)
    T = sum(q_lens)
    c = sink_case(q_lens, kv_lens, 8, Hkv, "BBND", gap, k=64, seed=103)
    c["blocks"][..., 0] = 0
    c["blocks"] = c["blocks"].sort(-1).values
    run(c, dev, sorted({0, T // 2, T - 1}))


def test_sink_in_the_middle_and_at_the_end(dev):
    """The largest score comes after the others: their sums are scaled down
    without being lost."""
    for q_lens, n in (([1], 20000), ([50], 20000)):
        for at in (9999, n - 51):
            run(sink_case(q_lens, [n], 8, 2, "BBND", 18.0, sink_at=at, seed=104), dev,
                (0, sum(q_lens) - 1))


def test_scores_that_climb(dev):
    """Every block's scores lie above those before it, by steps that move the
    running maximum each time, and by steps that it may lag."""
    for step in (0.3, 2.0, 9.0):
        for q_lens, kv, Hq in (([1], [2000], 8), ([90], [2000], 8), ([600], [700], 64)):
            c = lc.attention_case(q_lens, kv, Hq, 8 if Hq == 64 else 2, "BBND", FP, seed=105)
            c["q"] *= 0.25
            c["q"][..., 0] = AXIS
            for i in range(c["table"].shape[1]):
                c["k"][int(c["table"][0, i]), ..., 0] = i * step * math.sqrt(128) / AXIS
            log("climb", step, q_lens)
            run(c, dev, (0, sum(q_lens) - 1))
