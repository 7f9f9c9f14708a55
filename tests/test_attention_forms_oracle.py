"""The oracle's capped, biased and narrowed attention (oracle/layer.py) against
plain loops over one row at a time, against the plain attention where no form is
asked for, and on rows with a closed form."""
import math

import pytest
import torch

import layer_cases as lc
from oracle import layer

BF = torch.bfloat16


@pytest.mark.parametrize("layout", ["BBND", "BNBD", "TND"])
@pytest.mark.parametrize("mode", [0, 3])
def test_plain_is_the_plain_attention(layout, mode):
    c = lc.attention_case([3, 0, 70], [140, 5, 70], 6, 2, layout, BF, mode)
    args = (c["q"], c["k"], c["v"], c["table"], c["cu"], c["kv"], layout, mode)
    a, f = layer.attention(*args), layer.attention_forms(*args)
    assert torch.allclose(a.out, f.out, atol=1e-13) and torch.allclose(a.lse, f.lse, atol=1e-13)
    assert torch.allclose(a.spread, f.spread) and torch.equal(a.keys.double(), f.keys)
    assert torch.allclose(a.top, f.top)


@pytest.mark.parametrize("mode", [0, 3])
def test_row_by_row(mode):
    gen = torch.Generator().manual_seed(3)
    c = lc.attention_case([9, 2], [30, 140], 4, 2, "BBND", BF, mode)
    T = c["q"].shape[0]
    slopes = torch.tensor([0.5, 0.0, -0.1, 2.0])
    span = torch.randint(-5, 150, (T, 2), generator=gen).int()
    f = layer.attention_forms(c["q"] * 4, c["k"], c["v"], c["table"], c["cu"], c["kv"], "BBND",
                              mode, None, 3.0, slopes, span)
    for t, b, pos in layer.positions(c["cu"], c["kv"], T):
        for h in range(4):
            num, den, keys = torch.zeros(128, dtype=torch.float64), 0.0, 0
            for j in range(int(c["kv"][b])):
                if (mode == 3 and j > pos) or not int(span[t, 0]) <= j < int(span[t, 1]):
                    continue
                page, slot = int(c["table"][b, j // 128]), j % 128
                s = float(4 * c["q"][t, h].double() @ c["k"][page, slot, h // 2].double())
                s = 3 * math.tanh(s / math.sqrt(128) / 3) - float(slopes[h]) * abs(pos - j)
                num += math.exp(s) * c["v"][page, slot, h // 2].double()
                den, keys = den + math.exp(s), keys + 1
            assert int(f.keys[t, h]) == keys
            if keys:
                assert torch.allclose(f.out[t, h], num / den, rtol=1e-9, atol=1e-12)
                assert abs(float(f.lse[t, h]) - math.log(den)) < 1e-9
            else:
                assert not f.out[t, h].any() and float(f.lse[t, h]) == -math.inf


def test_closed_forms():
    """Equal keys: a cap leaves equal weights; a slope of ln 2 halves a key's
    weight with every step; a range of one key gives its value."""
    c = lc.attention_case([1], [5], 1, 1, "TND", torch.float32, 3)
    c["k"][:] = c["k"][0]
    args = (c["q"], c["k"], c["v"], None, c["cu"], c["kv"], "TND", 3)
    v = c["v"][:, 0].double()
    f = layer.attention_forms(*args, softcap=0.01)
    assert torch.allclose(f.out[0, 0], v.mean(0)) and abs(f.lse[0, 0] - math.log(5)) < 0.011
    f = layer.attention_forms(*args, slopes=torch.tensor([math.log(2.0)], dtype=torch.float64))
    w = torch.tensor([1.0, 2, 4, 8, 16], dtype=torch.float64) / 31
    assert torch.allclose(f.out[0, 0], w @ v)
    f = layer.attention_forms(*args, visible=torch.tensor([[2, 3]]))
    assert torch.allclose(f.out[0, 0], v[2]) and float(f.keys[0, 0]) == 1
