"""The layer oracle's own pins, on the CPU: its attention against torch's
float64 softmax written out over all keys, its append against closed forms, its
encoders against the formats' definitions; empty rows, bad pages and repeats."""
import math

import pytest
import torch

import layer_cases as lc
import oracle
from oracle import layer


def brute(c, blocks=None):
    """Full score matrix, masked, softmaxed, one request at a time."""
    T, Hq, _ = c["q"].shape
    Hkv = c["k"].shape[1 if c["layout"] != "BBND" else 2]
    out = torch.zeros(T, Hq, 128, dtype=torch.float64)
    first = 0
    for b, L in enumerate(c["kv"].tolist()):
        if c["layout"] == "TND":
            K, V = c["k"][first:first + L], c["v"][first:first + L]
        else:
            nb = -(-L // 128)
            pick = c["table"][b, :nb].long()
            K, V = (x[pick] if c["layout"] == "BBND" else x[pick].transpose(1, 2)
                    for x in (c["k"], c["v"]))
            K, V = (x.reshape(-1, Hkv, 128)[:L] for x in (K, V))
        first += L
        t0, t1 = int(c["cu"][b]), int(c["cu"][b + 1])
        q = c["q"][t0:t1].double()
        s = torch.einsum("qhd,khd->hqk", q, K.double().repeat_interleave(Hq // Hkv, 1))
        s = s / math.sqrt(128)
        pos = L - (t1 - t0) + torch.arange(t1 - t0)
        if c["mode"] == 3:
            s = s.masked_fill(torch.arange(L)[None] > pos[:, None], -math.inf)
        p = torch.softmax(s, -1).nan_to_num(0.0)
        out[t0:t1] = torch.einsum("hqk,khd->qhd", p, V.double().repeat_interleave(Hq // Hkv, 1))
    return out


@pytest.mark.parametrize("layout", ["TND", "BBND", "BNBD"])
@pytest.mark.parametrize("mode", [0, 3])
def test_attention_against_brute_force(layout, mode):
    c = lc.attention_case([3, 0, 9], [140, 20, 5], 4, 2, layout, torch.float16, mode)
    got = layer.attention(c["q"], c["k"], c["v"], c["table"], c["cu"], c["kv"], layout, mode)
    assert torch.allclose(got.out, brute(c), atol=1e-12)
    assert torch.equal(got.keys == 0, got.lse == -math.inf)


def test_selected_all_is_dense_and_none_is_empty():
    c = lc.attention_case([4], [300], 4, 2)
    args = (c["q"], c["k"], c["v"], c["table"], c["cu"], c["kv"], "BBND", 3, None)
    dense = layer.attention(*args)
    every = layer.attention(*args, torch.tensor([2, 0, 1, 1, -1, 99]).expand(4, 2, 6))
    none = layer.attention(*args, torch.full((4, 2, 3), -1))
    assert torch.equal(dense.out, every.out) and torch.equal(dense.lse, every.lse)
    assert (none.out == 0).all() and (none.lse == -math.inf).all()


def test_bad_pages_hide_their_keys():
    c = lc.attention_case([1], [300], 4, 2)
    c["table"][0, 1] = 10 ** 6
    got = layer.attention(c["q"], c["k"], c["v"], c["table"], c["cu"], c["kv"], "BBND", 0)
    assert (got.keys == 300 - 128).all()
    sel = layer.attention(c["q"], c["k"], c["v"], c["table"], c["cu"], c["kv"], "BBND", 0, None,
                          torch.tensor([0, 2]).expand(1, 2, 2))
    assert torch.allclose(got.out, sel.out, atol=1e-14)


def test_rotation_closed_forms():
    x = torch.randn(128, dtype=torch.float64)
    quarter = (torch.zeros(64), torch.ones(64))
    y, _ = layer.rotated(x, *quarter, False)
    assert torch.equal(y, torch.cat([-x[64:], x[:64]]))
    y, _ = layer.rotated(x, *quarter, True)
    assert torch.equal(y[0::2], -x[1::2]) and torch.equal(y[1::2], x[0::2])
    y, _ = layer.rotated(x, torch.zeros(8), torch.ones(8), False)
    assert torch.equal(y[16:], x[16:])
    a = torch.rand(64) * 6
    y, _ = layer.rotated(x, a.cos(), a.sin(), True)
    assert abs(float(y.norm() - x.norm())) < 1e-5


def test_encoders_against_the_oracles_decoders():
    """Every representable value encodes to itself, and what lies between goes
    to a neighbour."""
    for dt in (torch.float8_e4m3fn, torch.float8_e5m2):
        vals = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(dt)
        keep = torch.isfinite(vals.double())
        for part in vals.double()[keep].split(128):
            row = torch.zeros(128, dtype=torch.float64)
            row[:len(part)] = part
            got = oracle.decode(layer.encode_fp8(row, dt))
            assert torch.equal(torch.from_numpy(got), row)
        x = torch.randn(128, dtype=torch.float64) * 3
        assert torch.equal(layer.encode_fp8(x, dt).view(torch.uint8),
                           x.float().to(dt).view(torch.uint8))
    y = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6] * 16, dtype=torch.float64)
    y[32:64] *= -0.25
    code, scale = layer.encode_mxfp4(y)
    assert scale.tolist() == [127, 125, 127, 127]
    val = torch.from_numpy(oracle.decode(code)).view(4, 32)
    val = val * torch.exp2(scale.double() - 127)[:, None]
    assert torch.equal(val.flatten(), y)
    ties = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 4] * 16, dtype=torch.float64)
    val = torch.from_numpy(oracle.decode(layer.encode_mxfp4(ties)[0]))
    assert val[:8].tolist() == [0, 1, 1, 2, 2, 4, 4, 4]
    code, scale = layer.encode_i8(torch.linspace(-127, 127, 128, dtype=torch.float64))
    assert float(scale) == 1 and code[0] == -127 and code[-1] == 127
    for bad in (math.nan, math.inf):
        y[3] = bad
        assert math.isnan(float(layer.encode_i8(y)[1]))
        assert layer.encode_mxfp4(y)[1].tolist()[0] == 255


def test_append_places():
    cu, T = lc.lengths([2, 1])
    kv = torch.tensor([130, 1], dtype=torch.int32)
    table = torch.tensor([[4, 2], [0, -1]], dtype=torch.int32)
    src = torch.randn(T, 2, 128).to(torch.float16)
    for layout in ("BBND", "BNBD"):
        dst = torch.zeros(lc.cache_shape(layout, 5, 2), dtype=torch.float16)
        got = layer.append((src, dst, layout, None, False), None, None, table, cu, kv, False,
                           False)[0]
        at = (lambda p, s: got[p, s]) if layout == "BBND" else (lambda p, s: got[p, :, s])
        assert torch.equal(at(2, 0), src[0]) and torch.equal(at(2, 1), src[1])
        assert torch.equal(at(0, 0), src[2])
        assert int((got != 0).any(-1).sum()) == 6
    dst = torch.zeros(131, 2, 128, dtype=torch.float16)
    got = layer.append((src, dst, "TND", None, False), None, None, None, cu, kv, False, False)[0]
    assert torch.equal(got[128:131], src)
