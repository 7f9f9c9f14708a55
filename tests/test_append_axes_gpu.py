"""The cache append with several position axes: against the oracle
(oracle/layer.py), within half a step of the binary64 rotation and three float32
roundings (encoded rows bit for bit); and bit for bit against the append without
axes, by a table that holds each token's own angles."""
import sys

import pytest
import torch

import layer_cases as lc
from oracle import layer
from test_append_gpu import BF, FP, KINDS, angles, batch, bits, exact_dst, make_item

pytestmark = pytest.mark.gpu


def log(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import block_max_qk_amd
    block_max_qk_amd.load_library()
    return torch.device("cuda:0")


def pair_axes(half, axes, mix):
    if mix == "turns":
        return [r % axes for r in range(half)]
    return [r * axes // half for r in range(half)]


def call(items, cos, sin, table, cu, kv, dev, interleaved, axis_pos, pairs, **kw):
    import block_max_qk_amd as m
    put = lambda x: None if x is None else x.to(dev)  # noqa: E731
    live = [m.CacheItem(put(i[0]), put(i[1]), i[2], put(i[3]), i[4]) for i in items]
    m.msa_cache_append(live, put(cos), put(sin), put(table), put(cu), put(kv),
                       interleaved=interleaved, axis_positions=put(axis_pos), pair_axes=pairs,
                       **kw)
    torch.cuda.synchronize()
    return live


def check(items, cos, sin, table, cu, kv, dev, interleaved, axis_pos, pairs):
    live = call(items, cos, sin, table, cu, kv, dev, interleaved, axis_pos, pairs)
    rotated = any(i[4] for i in items)
    for i, d in zip(items, live):
        dst, scale, rows, mags, written = layer.append(i, cos, sin, table, cu, kv, interleaved,
                                                       rotated, axis_pos, pairs)
        got = d.dst.cpu()
        if got.element_size() == 1 or not i[4]:
            assert torch.equal(bits(got), bits(dst)), (i[2], i[1].dtype)
            assert scale is None or torch.equal(bits(d.scale.cpu()), bits(scale))
            continue
        info = torch.finfo(got.dtype)
        err = (got.double() - exact_dst(i, rows, written, table, cu, kv, cos)).abs()
        # two products and their sum in float32, then half a step of the type
        near = exact_dst(i, mags, written, table, cu, kv, cos) * 3 * 2.0 ** -24
        tol = near + (dst.double().abs() + near) * info.eps / 2 * 1.01
        tol = tol + info.smallest_normal * info.eps
        assert ((bits(got) == bits(dst)) | (err <= tol)).all(), float((err / tol).max())


@pytest.mark.parametrize("rot", [16, 48, 64, 128])
@pytest.mark.parametrize("pairs", ["halves", "interleaved"])
@pytest.mark.parametrize("axes,mix", [(1, "runs"), (2, "turns"), (3, "runs"), (3, "turns"),
                                      (4, "turns")])
def test_oracle(rot, pairs, axes, mix, dev):
    log("axes", rot, pairs, axes, mix)
    gen, cu, T, kv, table, pages = batch([3, 0, 5, 1], [260, 9, 5, 128], 60 + axes)
    cos, sin = angles(90, rot)          # fewer rows than positions
    ap = torch.randint(0, 90, (axes, T), generator=gen).int()
    src = torch.randn(T, 5, 128, generator=gen).to(FP if axes % 2 else BF)
    items = [make_item(src, k, lay, T, 5, pages, 0, gen, r)
             for k, lay, r in (("same", "BBND", True), ("e4m3", "BNBD", True),
                               ("i8", "BBND", True), ("mxfp4", "ROWS", True),
                               ("same", "ROWS", False))]
    check(items, cos, sin, table, cu, kv, dev, pairs == "interleaved", ap,
          pair_axes(rot // 2, axes, mix))


def test_any_map_of_the_pairs(dev):
    gen, cu, T, kv, table, pages = batch([7, 2], [7, 200], 70)
    for rot in (112, 128):
        cos, sin = angles(50, rot)
        ap = torch.randint(0, 50, (4, T), generator=gen).int()
        src = torch.randn(T, 2, 128, generator=gen).to(BF)
        pairs = torch.randint(0, 4, (rot // 2,), generator=gen).tolist()
        for il in (False, True):
            items = [make_item(src, "same", "BBND", T, 2, pages, 0, gen, True)]
            check(items, cos, sin, table, cu, kv, dev, il, ap, pairs)


def test_tokens_that_are_skipped(dev):
    """An axis outside the angle table, on any axis and in every item; the
    sequence's own position may lie past it.  Rows behind the last request and
    before the first are left."""
    gen, cu, T, kv, table, pages = batch([4, 3, 5], [2, 300, 200], 71, T_extra=4, first=1)
    cos, sin = angles(40, 64)
    ap = torch.randint(0, 40, (3, T), generator=gen).int()
    ap[0, 4], ap[1, 6], ap[2, 8], ap[2, 9] = 40, -1, 1 << 30, 39
    src = torch.randn(T, 2, 128, generator=gen).to(BF)
    items = [make_item(src, k, lay, T, 2, pages, 0, gen, r)
             for k, lay, r in (("same", "BBND", True), ("same", "BNBD", False),
                               ("same", "ROWS", True))]
    check(items, cos, sin, table, cu, kv, dev, False, ap, pair_axes(32, 3, "runs"))


@pytest.mark.parametrize("pairs", ["halves", "interleaved"])
@pytest.mark.parametrize("T", [1, 5, 3000])
def test_same_bits_as_angles_by_token(pairs, T, dev):
    """Long runs of steps too: an append whose table holds token t's own angles
    in row t gives the same bits."""
    gen, cu, _, kv, table, pages = batch([T], [T], 72)
    cos, sin = angles(500, 128)
    ap = torch.randint(0, 500, (3, T), generator=gen).int()
    axis = pair_axes(64, 3, "turns")
    at, r = ap.long()[axis].T, torch.arange(64)
    src = torch.randn(T, 40, 128, generator=gen).to(BF)
    one = src[:, :1].contiguous()
    mk = lambda: [make_item(src, "same", "BBND", T, 40, pages, 0, gen, True),  # noqa: E731
                  make_item(one, "e5m2", "BNBD", T, 1, pages, 0, gen, True),
                  make_item(one, "mxfp4", "ROWS", T, 1, pages, 0, gen, True)]
    a = mk()
    b = [[x.clone() if torch.is_tensor(x) else x for x in i] for i in a]
    got = call(a, cos, sin, table, cu, kv, dev, pairs == "interleaved", ap, axis)
    want = call(b, cos[at, r].contiguous(), sin[at, r].contiguous(), table, cu, kv, dev,
                pairs == "interleaved", None, None)
    for x, y in zip(got, want):
        assert torch.equal(bits(x.dst), bits(y.dst))


def test_captured_and_replayed(dev):
    """Axis positions are read by each replay."""
    import block_max_qk_amd as m
    gen, cu, T, kv, table, pages = batch([6], [6], 73)
    cos, sin = (x.to(dev) for x in angles(30, 128))
    src = torch.randn(T, 4, 128, generator=gen).to(BF).to(dev)
    out, eager = torch.zeros_like(src), torch.zeros_like(src)
    ap = torch.zeros(3, T, dtype=torch.int32, device=dev)
    cu, kv = cu.to(dev), kv.to(dev)
    axis = bytes(pair_axes(64, 3, "runs"))

    def step(dst):
        m.msa_cache_append([m.CacheItem(src, dst, "ROWS", rotate=True)], cos, sin, None, cu, kv,
                           axis_positions=ap, pair_axes=axis)

    step(eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    for i in range(4):
        ap.copy_(torch.randint(0, 30, (3, T), generator=gen).int())
        step(eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_kinds_of_integers(dev):
    """The pairs' axes as bytes, lists, arrays and tensors of any integers."""
    import numpy as np
    gen, cu, T, kv, table, pages = batch([4, 1], [4, 1], 75)
    cos, sin = angles(30, 64)
    src = torch.randn(T, 2, 128, generator=gen).to(BF)
    ap = torch.randint(0, 30, (3, T), generator=gen).int()
    axis = pair_axes(32, 3, "turns")
    b = [[src, torch.zeros_like(src), "ROWS", None, True]]
    want = call(b, cos, sin, None, cu, kv, dev, False, ap, axis)[0].dst
    assert not torch.equal(want.cpu(), call(b, cos, sin, None, cu, kv, dev, False, ap,
                                            [0] * 32)[0].dst.cpu())
    for pairs in (bytes(axis), bytearray(axis), tuple(axis), np.array(axis, np.int32),
                  np.array(axis, np.uint8), torch.tensor(axis)):
        got = call(b, cos, sin, None, cu, kv, dev, False, ap, pairs)[0].dst
        assert torch.equal(got, want), type(pairs)


def test_refusals(dev):
    import block_max_qk_amd as m
    gen, cu, T, kv, table, pages = batch([4], [4], 74)
    cos, sin = (x.to(dev) for x in angles(30, 64))
    src = torch.randn(T, 2, 128, generator=gen).to(BF).to(dev)
    ap = torch.zeros(3, T, dtype=torch.int32, device=dev)
    good = [0, 1, 2, 2] * 8

    def go(ap=ap, pairs=good):
        m.msa_cache_append([m.CacheItem(src, src.clone(), "ROWS", rotate=True)], cos, sin, None,
                           cu.to(dev), kv.to(dev), axis_positions=ap, pair_axes=pairs)

    go()
    for kw in (dict(ap=ap.long()), dict(ap=ap[:, :3]), dict(ap=ap[0]), dict(ap=ap.cpu()),
               dict(ap=None), dict(pairs=None), dict(pairs=good[:-1]), dict(pairs=[-1] * 32),
               dict(pairs=[300] * 32), dict(pairs=[0.5] * 32)):
        with pytest.raises(ValueError):
            go(**kw)
    for kw in (dict(pairs=[3] * 32), dict(ap=torch.zeros(5, T, dtype=torch.int32, device=dev)),
               dict(ap=torch.zeros(0, T, dtype=torch.int32, device=dev))):
        with pytest.raises(m.MsaError):
            go(**kw)
