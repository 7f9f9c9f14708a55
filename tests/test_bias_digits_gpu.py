"""Biased scores of tokens that see far keys only: what all of a row's keys have in
common of their biases costs none of their weights' digits, within the oracle's
bounds (oracle/layer.py), which take the bias relative to the nearest key's."""
import pytest
import torch

from test_attention_forms_gpu import BF, FP, call, check, dev, make, pos_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,cap", [(BF, 0.0), (FP, 0.0), (BF, 20.0)])
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv", [
    ([1, 1], [30000, 9000], 4, 1), ([40], [30000], 8, 2), ([130, 3], [12000, 30000], 4, 1),
    ([2, 30], [400, 20000], 4, 4)])
def test_far_keys_only(q_lens, kv_lens, Hq, Hkv, dtype, cap, dev):
    """Ranges before the token (their last keys the nearest), and without a causal mask
    behind it too; whole, split and joined."""
    for mode in (3, 0):
        c = make(q_lens, kv_lens, Hq, Hkv, "BNBD", dtype, mode, cap, gain=2.0)
        c["slopes"] = torch.tensor([0.7, 0.31, 0.011, 3.3, -0.2, 0.0, 17.0, 0.1])[:Hq].contiguous()
        pos = pos_of(c)
        ranges = [(pos * 0, pos * 0 + 200), (pos // 2 - 70, pos // 2 + 1),
                  (pos * 0 + 100, pos - 300)]
        if mode == 0:
            ranges += [(pos + 1, pos + 150)]
        for first, end in ranges:
            c["visible"] = torch.stack([first, end], 1).int()
            print("far keys", q_lens, mode, dtype, cap, int(first[0]), flush=True)
            check(c, *call(c, dev))


def test_no_keys_and_no_pages(dev):
    """Rows that see nothing, and rows whose nearest keys lie on no page."""
    c = make([1, 40], [900, 2000], 4, 2, bias=True)
    pos = pos_of(c)
    c["visible"] = torch.stack([pos * 0 + 10, pos - 200], 1).int()
    c["visible"][5::7] = 0
    c["table"][1, 12] = c["table"][1, 13] = c["table"][0, 4] = -1
    check(c, *call(c, dev))


def test_tokens_before_all_keys(dev):
    """More new tokens than keys, without a causal mask: positions below 0."""
    c = make([9, 200], [4, 150], 8, 2, mode=0, bias=True)
    c["visible"] = torch.tensor([[20, 140]], dtype=torch.int32).expand(209, 2).contiguous()
    check(c, *call(c, dev))


@pytest.mark.parametrize("Hq,Hkv,q_lens,kv_lens", [
    (32, 1, [8], [320]), (8, 2, [70], [448]), (64, 1, [2, 3], [192, 256])])
def test_steep_heads(Hq, Hkv, q_lens, kv_lens, dev):
    """A token's own key is off by none of its neighbours' biases, also where it ends a
    stage of keys that all rows see whole: the last of 64."""
    c = make(q_lens, kv_lens, Hq, Hkv, "BNBD", BF, gain=1.0, bias=True)
    c["slopes"] = torch.linspace(37.7, 30011.3, Hq)
    assert (pos_of(c) % 64 == 63).any()
    check(c, *call(c, dev))
    c["visible"] = torch.stack([pos_of(c) * 0, pos_of(c) - 64], 1).int()
    check(c, *call(c, dev))


@pytest.mark.parametrize("q_lens,kv_lens,cap", [([1], [130], 0.0), ([90], [300], 0.0),
                                                ([90], [300], 9.0)])
def test_the_steepest_slopes(q_lens, kv_lens, cap, dev):
    """Slopes whose product with 1 / softmax_scale has no float32 leave each token its
    own key alone: its value, and its score as lse."""
    c = make(q_lens, kv_lens, 4, 2, "TND", BF, cap=cap)
    c["slopes"] = torch.tensor([3.4e38, 1e38, 2.6e38, 4e37])
    out, lse = call(c, dev)
    own = pos_of(c)
    k, v = (c[n][own].repeat_interleave(2, 1).double() for n in ("k", "v"))
    assert torch.equal(out.double(), v)
    s = (c["q"].double() * k).sum(-1) * 128 ** -0.5
    size = (c["q"].double() * k).abs().sum(-1) * 128 ** -0.5
    if cap:
        s = cap * torch.tanh(s / cap)
    e = 2.0 ** -24
    assert ((lse.double() - s).abs() <= 130 * e * size + 12 * e * cap + 8 * e * (1 + s.abs())).all()


@pytest.mark.parametrize("n", [1, 40])
def test_positions_past_2_to_the_24(n, dev):
    """Only the distances count: keys near the end of a context of 2^25 tokens (a table
    that names few pages many times) give the bits of a short context's."""
    import block_max_qk_amd as m
    gen = torch.Generator().manual_seed(n)
    k, v = torch.randn(2, 8, 128, 1, 128, generator=gen).to(BF).to(dev)
    q = torch.randn(n, 4, 128, generator=gen).to(BF).to(dev)
    slopes = torch.tensor([0.5, 0.01, -0.1, 3.0], device=dev)
    cu = torch.tensor([0, n], dtype=torch.int32, device=dev)
    got = []
    for blocks in (8, (1 << 18) + 8):
        kv = blocks * 128 - 5
        table = torch.arange(blocks, dtype=torch.int32, device=dev)[None] % 8
        first = kv - 700
        visible = torch.tensor([[first, kv - 60 - n]], dtype=torch.int32, device=dev)
        got.append(m.attention(q, k, v, table, cu, torch.tensor([kv], dtype=torch.int32,
                                                                device=dev),
                               "BBND", return_lse=True, slopes=slopes,
                               visible=visible.expand(n, 2).contiguous()))
    torch.cuda.synchronize()
    (a, al), (b, bl) = got
    # (the parts may be split elsewhere: sums in another order and weights rounded to 16
    # bits against another power of two, half a step of each and of the results)
    tol = 2.0 ** -20 * (1 + al.abs())
    assert ((al - bl).abs() <= tol).all(), float((al - bl).abs().max())
    assert ((a.float() - b.float()).abs() <= 2.0 ** -7 * a.float().abs() + 2.0 ** -8).all()
