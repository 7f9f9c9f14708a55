"""Capped scores to their own last digits: over a single key the log of the
softmax's sum is the capped score itself (over 128 equal keys ln 128 more), and a
query and a key of one non-zero element each make an exact product.

With e = 2^-24 a capped score is off by at most 8 e of itself (below 5/8 of the
cap 2.1 e of the polynomial's fit, 1 e each of its first coefficient, its last sum
and the product, 0.5 e of the smaller terms; above it 2.9 e of the cap, at
0.55 of it, of the exponential and the reciprocal, 1 e each of the cap and the last
sum), and the log of the sum by 4 e (1 + |score|), e for each key, and 24 e where
float16's lift (2^11) is added and taken off."""
import math
import sys

import pytest
import torch

from test_attention_forms_gpu import call, make, reference
from test_attention_forms_gpu import check as check_forms

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
E = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_max_qk_amd
    block_max_qk_amd.load_library()
    return torch.device("cuda:0")


KEYS = {"rows": 1, "tiles": 1, "stages": 128}


def capped(s, cap, scale, kernel, dtype, dev, key=1.0):
    """lse of queries s (and a key) over one key each: many requests of one token (16
    rows a tile), or one of many tokens (128 rows), whose stage is not whole; or over
    two whole stages of equal keys, ln 128 taken off."""
    import block_max_qk_amd as m
    n, keys = len(s), KEYS[kernel]
    q = torch.zeros(n, 1, 128, dtype=dtype)
    q[:, 0, 5] = s
    k = torch.zeros(n if kernel == "rows" else keys, 1, 128, dtype=dtype)
    k[:, 0, 5] = key
    ints = dict(dtype=torch.int32, device=dev)
    if kernel == "rows":
        cu, kv = torch.arange(n + 1, **ints), torch.ones(n, **ints)
    else:
        cu, kv = torch.tensor([0, n], **ints), torch.tensor([keys], **ints)
    want = 16 if kernel == "rows" else 128
    assert m.msa_attention_tile_rows(n, len(kv), 1, 1, 1) == want
    print("capped", cap, kernel, dtype, file=sys.stderr, flush=True)
    _, lse = m.attention(q.to(dev), k.to(dev), k.to(dev), None, cu, kv, "TND", 0, scale,
                         max_blocks=1, return_lse=True, softcap=cap)
    torch.cuda.synchronize()
    return lse.cpu()[:, 0].double() - math.log(keys)


def sweep(cap, scale, parts, dtype):
    """Queries whose scores are these parts of the cap, of either sign."""
    s = (parts * (cap / scale)).to(dtype)
    return torch.cat([s, -s])


def check(got, s, cap, scale, kernel, dtype):
    want = cap * torch.tanh(s.double() * scale / cap)
    n = KEYS[kernel]
    tol = (8 * E * want.abs() + 4 * E * (1 + math.log(n) + want.abs()) + (n - 1) * E
           + (24 * E if dtype == FP else 0))
    err = (got - want).abs()
    at = int((err / tol).nan_to_num(1e30).argmax())
    assert (err <= tol).all(), (float((err / tol).max()), float(s[at] * scale / cap))


NEAR = torch.logspace(-3, -0.30103, 300, dtype=torch.float64)       # to half the cap


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kernel", ["rows", "tiles", "stages"])
def test_below_the_cap(kernel, dtype, dev):
    """Waves whose scores all stay below half the cap."""
    for cap, scale in ((50.0, 0.125), (1000.0, 0.125), (1000.0, 1.0)):
        s = sweep(cap, scale, NEAR, dtype)
        check(capped(s, cap, scale, kernel, dtype, dev), s, cap, scale, kernel, dtype)


@pytest.mark.parametrize("kernel", ["rows", "tiles", "stages"])
def test_caps_of_any_size(kernel, dev):
    """Caps whose polynomial has no float32 coefficients without a scaling of its
    argument: large ones, whose scores are ordinary or near them, and small ones."""
    for cap in (2000.0, 2200.0, 1e4, 1e5, 1e7, 1e12, 1e20, 1e30, 1e-4, 1e-12):
        for low in (-1.0, -4.0, -7.0):
            s = sweep(cap, 0.125, torch.logspace(low, low + 0.7, 200, dtype=torch.float64), BF)
            check(capped(s, cap, 0.125, kernel, BF, dev), s, cap, 0.125, kernel, BF)
    s = torch.logspace(-1, 3, 400, dtype=torch.float64).to(BF)      # ordinary scores
    for cap in (1e4, 1e5, 1e7, 1e30):
        check(capped(s, cap, 0.125, kernel, BF, dev), s, cap, 0.125, kernel, BF)


@pytest.mark.parametrize("kernel", ["rows", "tiles", "stages"])
def test_caps_next_to_the_types_end(kernel, dev):
    """Twice the cap in units of log2 has no float32."""
    for cap in (1e38, 2e38):
        s = (torch.tensor([0.7, -1.1, 0.9, 1.5] * 10).double() * (cap * 2.0 ** -63)).to(BF)
        s1 = s.double() * 2.0 ** 63
        check(capped(s, cap, 1.0, kernel, BF, dev, 2.0 ** 63), s1, cap, 1.0, kernel, BF)
        s = torch.tensor([1.0, -3.0, 1e5, 1e9, -1e12, 1e15]).to(BF).repeat(10)
        for key in (1.0, 2.0 ** 33, 2.0 ** 60):
            s1 = s.double() * key
            check(capped(s, cap, 1.0, kernel, BF, dev, key), s1, cap, 1.0, kernel, BF)


@pytest.mark.parametrize("kernel", ["rows", "tiles", "stages"])
def test_scores_of_any_size(kernel, dev):
    """Scores whose rounding is more than an exponent holds: the largest weighs 1."""
    for cap in (1e10, 1e12):
        s = sweep(cap, 1e6, torch.logspace(-4, -0.31, 100, dtype=torch.float64), BF)
        check(capped(s, cap, 1e6, kernel, BF, dev), s, cap, 1e6, kernel, BF)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 2], [200, 130]), ([60], [200]), ([40], [3333])])
def test_caps_far_above_the_scores(q_lens, kv_lens, dev):
    """Ordinary scores under a huge cap are the uncapped ones, within their bounds (with
    cap = 10^6 and scores of 100 a cap takes 10^-8 of a score off it, less than a tenth
    of what the bounds hold)."""
    for gain in (0.01, 1.0, 10.0):
        c = make(q_lens, kv_lens, 8, 2, gain=gain)
        want = reference(c)
        for cap in (1e6, 1e7, 1e12, 1e30):
            check_forms({**c, "cap": cap}, *call({**c, "cap": cap}, dev), want)
