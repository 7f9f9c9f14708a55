"""A row's bits do not depend on the rows that share its tile, nor on keys that it
does not see: with plain, biased and narrowed scores, in tiles of 16, 128 and 256
rows that are not split.  (Capped scores go by the largest beside them.)"""
import sys

import pytest
import torch

from test_attention_forms_gpu import BF, FP, call, dev, make, pos_of  # noqa: F401

pytestmark = pytest.mark.gpu

FORMS = [{}, dict(bias=True), dict(bias=True, mode=0), dict(mask="documents"),
         dict(bias=True, mask="documents"), dict(bias=True, mask="any")]


def same(a, b, rows=slice(None)):
    assert all(torch.equal(x[rows], y[rows]) for x, y in zip(a, b))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,dtype,width", [
    ([2], [300], 8, 1, BF, None), ([4, 3], [200, 140], 4, 1, FP, None),     # 16 rows
    ([50], [300], 8, 2, BF, None), ([90, 70], [90, 400], 2, 2, FP, None),   # 128 rows
    ([700, 900], [700, 1000], 32, 16, BF, 130),                             # 256 rows
])
def test_other_rows_queries(form, q_lens, kv_lens, Hq, Hkv, dtype, width, dev):
    print("queries", form, q_lens, file=sys.stderr, flush=True)
    c = make(q_lens, kv_lens, Hq, Hkv, "BBND", dtype, gain=1.0, seed=4, width=width, **form)
    want = call(c, dev)
    T = len(c["q"])
    for factor in (40.0, 0.0):
        for other in (torch.arange(T) % 3 == 1, torch.arange(T) >= T - 1):
            d = {**c, "q": c["q"].clone()}
            d["q"][other] *= factor
            same(call(d, dev), want, ~other)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("lens,dtype", [((20, 29, 50), BF), ((60, 61, 97), FP)])
def test_other_tokens_beside_it(form, lens, dtype, dev):
    """The last tokens of a request, with other numbers of tokens before them."""
    got = []
    for n in lens:
        c = make([n], [300], 8, 2, "BBND", dtype, gain=1.0, seed=6, **form)
        if not got:
            first = c
        keep = lens[0]
        # the same queries, keys and ranges, and others in front
        d = {**c, "q": c["q"].clone(), "k": first["k"], "v": first["v"], "table": first["table"]}
        d["q"][n - keep:] = first["q"]
        if form.get("mask"):
            d["visible"] = c["visible"].clone()
            d["visible"][n - keep:] = first["visible"]
        got.append([x[n - keep:] for x in call(d, dev)])
    for x in got[1:]:
        same(x, got[0])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv", [([2], [300], 8, 1), ([100], [300], 8, 2)])
def test_keys_that_it_does_not_see(form, q_lens, kv_lens, Hq, Hkv, dev):
    c = make(q_lens, kv_lens, Hq, Hkv, "TND", BF, gain=1.0, **form)
    pos = pos_of(c)
    if c["visible"] is not None:
        c["visible"] = torch.stack([(pos - 60).clamp(min=0), pos + 1], 1).int()
    j = kv_lens[0] - 1
    sees = pos >= j if c["mode"] == 3 else torch.ones(len(pos), dtype=torch.bool)
    want = call(c, dev)
    for factor in (1e3, -1e3, 0.0):
        d = {**c, "k": c["k"].clone(), "v": c["v"].clone()}
        d["k"][j] *= factor
        d["v"][j] *= factor
        same(call(d, dev), want, ~sees)
