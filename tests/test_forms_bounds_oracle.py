"""The bounds of the capped attention's tests are of use: results of other scores than
the call's lie outside them, whatever the cap's size."""
import pytest
import torch

from oracle import layer
from test_attention_forms_gpu import check, make, reference


def refused(c, wrong):
    """Whether the check of the GPU tests refuses results of the scores of `wrong`."""
    f = reference(wrong)
    try:
        check(c, f.out.to(c["q"].dtype), f.lse.float(), reference(c))
    except AssertionError:
        return True
    return False


@pytest.mark.parametrize("cap", [8.0, 1e4, 1e5, 1e7, 1e30])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 2], [200, 130]), ([60], [200])])
def test_scores_left_out(q_lens, kv_lens, cap):
    for gain in (0.01, 3.0):
        c = make(q_lens, kv_lens, 8, 2, cap=cap, gain=gain)
        assert not refused(c, c)
        assert refused(c, {**c, "q": c["q"] * 0})
    if cap > 8:                       # scores off by 2^-9 of themselves
        c = make(q_lens, kv_lens, 8, 2, cap=cap, gain=40.0)
        assert refused(c, {**c, "scale": 128 ** -0.5 * (1 + 2.0 ** -9)})


@pytest.mark.parametrize("cap", [1e5, 1e7])
def test_large_scores_left_out(cap):
    for part in (0.02, 0.2, 0.6):
        c = make([60], [200], 8, 2, gain=1.0)
        top = reference({**c, "cap": 0.0}).lse.max()
        c["q"] = (c["q"].float() * float(part * cap / top)).to(c["q"].dtype)
        c["cap"] = cap
        assert not refused(c, c)
        assert refused(c, {**c, "q": c["q"] * 0})
