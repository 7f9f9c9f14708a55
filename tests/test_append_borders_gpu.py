"""fp8 rows whose rotated value lies next to the border between two codes, too
near for a float32 to tell: each falls on its own side."""
import sys

import pytest
import torch

import layer_cases as lc
from test_append_gpu import batch, make_item, run

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_max_qk_amd
    block_max_qk_amd.load_library()
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kind,lower,step", [("e4m3", 1.5, 0.125), ("e4m3", 1.625, 0.125),
                                             ("e5m2", 1.0, 0.25), ("e5m2", 1.25, 0.25)])
@pytest.mark.parametrize("pairs", ["halves", "interleaved"])
def test_a_hair_past_a_tie(dtype, kind, lower, step, pairs, dev):
    """Pairs (1, 1) with cosine `middle` and sine +-2^-30: a' = middle - s lies a
    hair below or above the middle of two codes, b' = middle + s on the other
    side; and the same of (-1, -1) and far smaller, with a tie exactly between."""
    print("borders", kind, lower, pairs, file=sys.stderr, flush=True)
    gen, cu, T, kv, table, pages = batch([4], [4], 51)
    middle = lower + step / 2
    cos = torch.full((4, 64), middle)
    sin = torch.zeros(4, 64)
    sin[0], sin[1] = 2.0 ** -30, -2.0 ** -30
    sin[3] = 2.0 ** -30 * torch.where(torch.arange(64) % 3 > 0, 1.0, -1.0)
    src = torch.ones(T, 2, 128)
    src[:, 1] = -2.0 ** -4
    src = src.to(dtype)
    items = [make_item(src, kind, layout, T, 2, pages, 0, gen, True) for layout in ("BBND", "ROWS")]
    live = run(items, cos, sin, table, cu, kv, dev, pairs == "interleaved")
    # the codes by hand: below the middle the lower one, above it the upper
    rows = live[1].dst.cpu().double()
    a, b = ((slice(0, 64), slice(64, 128)) if pairs == "halves" else
            (slice(0, 128, 2), slice(1, 128, 2)))
    for h, unit in ((0, 1.0), (1, -2.0 ** -4)):
        assert (rows[0, h, a] == unit * lower).all()
        assert (rows[0, h, b] == unit * (lower + step)).all()
        assert (rows[1, h, a] == unit * (lower + step)).all()
        assert (rows[1, h, b] == unit * lower).all()
        # a tie goes to the code with an even last bit
        even = lower if (lower / step) % 2 == 0 else lower + step
        assert (rows[2, h] == unit * even).all()


def test_an_ordinary_rotation_next_to_a_border(dev):
    """a c - b s = 1.5625 + 2^-26.7 for angles near 4.07 radians."""
    gen, cu, T, kv, table, pages = batch([1], [1], 52)
    c = torch.tensor(-0.600007951, dtype=torch.float32)
    s = torch.tensor(-0.799994051, dtype=torch.float32)
    src = torch.zeros(1, 1, 128)
    src[..., :64], src[..., 64:] = -0.9375, 1.25
    y = -0.9375 * c.double() - 1.25 * s.double()
    assert 1.5625 < float(y) < 1.5625 + 2.0 ** -24 and float(y.float()) == 1.5625
    items = [make_item(src.to(BF), "e4m3", "ROWS", 1, 1, pages, 0, gen, True)]
    live = run(items, c.expand(1, 64).contiguous(), s.expand(1, 64).contiguous(), table, cu, kv, dev)
    assert (live[0].dst.cpu().float()[..., :64] == 1.625).all()


def test_values_past_float32_and_below_it(dev):
    """Rotated rows past the largest float32 stay at the format's largest value,
    rows far below its smallest step give zeros of their sign."""
    gen, cu, T, kv, table, pages = batch([3], [3], 53)
    cos, sin = torch.full((3, 64), 0.75), torch.full((3, 64), -0.75)
    src = torch.zeros(3, 1, 128)
    src[0] = 3e38
    src[1] = -1e-38
    src[2] = 2.0 ** -12
    for kind in ("e4m3", "e5m2"):
        items = [make_item(src.to(BF), kind, "ROWS", T, 1, pages, 0, gen, True)]
        live = run(items, cos, sin, table, cu, kv, dev)
        got = live[0].dst.cpu().float()[0, 0]
        assert (got[:64] == (448 if kind == "e4m3" else 57344)).all() and (got[64:] == 0).all()
