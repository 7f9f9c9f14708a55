"""The step tables' entry on the CPU: every malformed call is rejected with its
status before anything is launched (no call here is valid), and the oracle's
figures on a step worked by hand."""
import torch

import block_max_qk_amd as m
from oracle import layer

OK, NULL, LAYOUT, DTYPE, SHAPE, STRIDE = range(6)
# addresses far apart, never dereferenced
AT = {n: 0x100000 * (i + 1) for i, n in enumerate(
    ("new", "ctx", "rows", "pool", "free", "count", "left", "cu", "kv", "start", "table", "pos",
     "slots", "pages"))}


def call(B=2, R=4, W=8, F=10, MB=8, T=16, bs=128, **kw):
    a = {**AT, **kw}
    return m.load_library().msa_step_tables(
        a["new"], a["ctx"], a["rows"], B, a["pool"], R, W, a["free"], F, a["count"], a["left"], MB,
        T, bs, a["cu"], a["kv"], a["start"], a["table"], a["pos"], a["slots"], a["pages"], None)


def test_nulls():
    for n in AT:
        if n != "rows":
            assert call(**{n: None}) == NULL, n


def test_sizes():
    for kw in (dict(B=-1), dict(B=(1 << 20) + 1), dict(B=(1 << 30) + 1),
               dict(R=(1 << 31) - 1, W=(1 << 31) - 1), dict(T=-1), dict(T=1 << 31), dict(bs=64),
               dict(MB=0), dict(MB=9), dict(MB=(1 << 24) + 1, W=1 << 25), dict(R=-1),
               dict(R=1 << 31), dict(W=1 << 31), dict(F=-1), dict(F=1 << 31)):
        assert call(**kw) == SHAPE, kw


def test_alignment():
    for n in AT:
        assert call(**{n: AT[n] + 2}) == STRIDE, n
    assert call(slots=AT["slots"] + 4) == STRIDE


def test_overlaps():
    written = ("pool", "cu", "kv", "start", "table", "pos", "slots", "pages", "left")
    for w in written:
        for other in ("new", "ctx", "rows", "free", *written):
            if other != w:
                assert call(**{w: AT[other]}) == STRIDE, (w, other)
        if w != "left":
            assert call(**{w: AT["count"]}) == STRIDE, w
    # the end of one array in another
    assert call(kv=AT["ctx"] + 4) == STRIDE
    assert call(ctx=AT["table"] + 4 * 2 * 8 - 4) == STRIDE
    assert call(left=AT["pages"] + 8) == STRIDE


def test_oracle_by_hand():
    """Two requests: 130 tokens in an empty row take two pages; 3 tokens behind
    127 fill the first block and begin the second."""
    pool = torch.full((3, 3), -1, dtype=torch.int32)
    pool[0, 0] = 4
    got = layer.step_tables([130, 3], [0, 127], [2, 0], pool, [9, 8, 7, 6, 5], 4, 3, 135)
    assert got["cu_seqlens_q"] == [0, 130, 133]
    assert got["kv_len"] == [130, 130] and got["start_loc"] == [0, 0]
    assert got["cu_pages"] == [0, 2, 3] and got["free"] == [1, 0]
    assert got["block_table"].tolist() == [[6, 7, -1], [4, 8, -1]]
    assert got["pool"].tolist() == [[4, 8, -1], [-1, -1, -1], [6, 7, -1]]
    assert got["positions"] == [*range(130), 127, 128, 129, 0, 0]
    assert got["slots"][:130] == [*range(768, 896), 896, 897]
    assert got["slots"][130:] == [4 * 128 + 127, 8 * 128, 8 * 128 + 1, -1, -1]
    # one page left: the second block goes without
    got = layer.step_tables([130], [0], None, pool.clone().fill_(-1), [3], 1, 3, 130)
    assert got["block_table"].tolist() == [[3, -1, -1]] and got["free"] == [0, 1]
    assert got["slots"][127:] == [3 * 128 + 127, -1, -1]


def test_refused_off_the_gpu():
    """(index -1: the binding refuses tensors in host memory)"""
    out = m.new_step_tables(1, 2, 2)
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    try:
        m.msa_step_tables(i32(1), i32(1), i32(2, 2), i32(4), i32(2), out)
    except ValueError as e:
        assert "GPU" in str(e)
    else:
        raise AssertionError("host tensors were taken")
