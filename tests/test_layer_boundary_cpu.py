"""The cache append and the attention on the CPU: every malformed call is
rejected with its status (or the binding's error) before anything is launched,
and the workspace sizes hold together.  No call here reaches a launch: each
fails validation or has T = 0."""
import ctypes
import struct

import pytest
import torch

import block_max_qk_amd as m
from block_max_qk_amd._binding import MsaTensor

OK, NULL, LAYOUT, DTYPE, SHAPE, STRIDE, SCALE, ATTR, HIP, WORKSPACE = range(10)
TND, BBND, BNBD, ROWS = 0, 1, 2, 3
F16, BF16, I8, E4M3, E5M2, MX = range(6)
FAKE = 0x10000          # never dereferenced
ITEM = struct.Struct("<Qii4q4qQii4q4qQii")       # msa_append_item_t


def desc(shape, stride=None, dtype=F16, addr=FAKE):
    d = MsaTensor()
    d.data, d.dtype, d.ndim = addr, dtype, len(shape)
    if stride is None:
        stride, n = [], 1
        for x in reversed(shape):
            stride.insert(0, n)
            n *= x
    for i, (x, y) in enumerate(zip(shape, stride)):
        d.shape[i], d.stride[i] = x, y
    return d


def attend(q=None, k=None, v=None, *, table=FAKE, mb=4, cu=FAKE, kv=FAKE, B=1, bs=128,
           layout=BBND, mode=3, scale=0.1, out=FAKE, lse=None, ws=None, wb=0, blocks=None, n=0,
           T=0):
    lib = m.load_library()
    q = desc((T, 8, 128)) if q is None else q
    k = desc((6, 128, 2, 128)) if k is None else k
    v = desc((6, 128, 2, 128)) if v is None else v
    head = [None if x == "null" else ctypes.byref(x) for x in (q, k, v)]
    tail = [table, mb, cu, kv, B, bs, layout, mode, scale, out, lse, ws, wb, None]
    if n:
        return lib.msa_block_attention(*head, blocks, n, *tail)
    return lib.msa_attention(*head, *tail)


def test_valid_empty_calls_return_ok():
    assert attend() == OK
    assert attend(n=16) == OK
    assert attend(B=0, cu=FAKE, kv=None, table=None) == OK
    assert attend(k=desc((0, 2, 128), addr=None), v=desc((0, 2, 128), addr=None), layout=TND,
                  table=None) == OK
    assert attend(k=desc((6, 128, 128)), v=desc((6, 128, 128))) == OK       # one head, no axis


def test_attention_nulls():
    assert attend(q="null") == NULL
    assert attend(k="null") == NULL
    assert attend(v="null") == NULL
    assert attend(cu=None) == NULL
    assert attend(kv=None) == NULL
    assert attend(table=None) == NULL
    assert attend(T=2, out=None) == NULL
    assert attend(T=2, n=4, blocks=None) == NULL


def test_attention_data_nulls():
    none = desc((6, 128, 2, 128), addr=None)
    assert attend(q=desc((2, 8, 128), addr=None), T=2) == NULL
    assert attend(k=none, T=2) == NULL
    assert attend(v=none, T=2) == NULL
    assert attend(v=none, T=2, n=4, blocks=FAKE) == NULL


@pytest.mark.parametrize("layout", [-1, 3, 7])
def test_attention_layouts(layout):
    assert attend(layout=layout) == LAYOUT


def test_attention_types():
    for dt in (I8, E4M3, E5M2, MX, 9):
        assert attend(q=desc((0, 8, 128), dtype=dt)) == DTYPE
    assert attend(k=desc((6, 128, 2, 128), dtype=BF16)) == DTYPE
    assert attend(v=desc((6, 128, 2, 128), dtype=BF16)) == DTYPE


def test_attention_shapes():
    for q in ((0, 8), (0, 8, 64), (0, 7, 128), (0, 0, 128)):
        assert attend(q=desc(q)) == SHAPE, q
    for k in ((6, 64, 2, 128), (6, 128, 2, 64), (0, 128, 2, 128), (6, 128)):
        assert attend(k=desc(k)) == SHAPE, k
    assert attend(v=desc((5, 128, 2, 128))) == SHAPE
    assert attend(v=desc((6, 128, 4, 128))) == SHAPE
    assert attend(bs=64) == SHAPE
    assert attend(mb=0) == SHAPE
    assert attend(mb=1 << 25) == SHAPE
    assert attend(B=-1) == SHAPE
    assert attend(B=0, T=2) == SHAPE
    assert attend(layout=TND, k=desc((9, 2, 128)), v=desc((9, 2, 128))) == SHAPE   # with a table


def test_attention_strides():
    assert attend(q=desc((2, 8, 128), (1024, 256, 1)), T=2) == STRIDE
    assert attend(q=desc((2, 8, 128), (1024, 128, 2)), T=2) == STRIDE
    assert attend(q=desc((2, 8, 128), (512, 128, 1)), T=2) == STRIDE
    assert attend(q=desc((2, 8, 128), (1028, 128, 1)), T=2) == STRIDE
    assert attend(q=desc((0, 8, 128), addr=FAKE + 8)) == STRIDE
    assert attend(k=desc((6, 128, 2, 128), (32768, 256, 64, 1))) == STRIDE
    assert attend(k=desc((6, 128, 2, 128), (32764, 256, 128, 1))) == STRIDE
    assert attend(k=desc((6, 128, 2, 128), (0, 256, 128, 1))) == STRIDE
    assert attend(v=desc((6, 128, 2, 128), addr=FAKE + 4)) == STRIDE
    assert attend(out=FAKE + 2) == STRIDE
    assert attend(lse=FAKE + 2) == STRIDE
    assert attend(ws=FAKE + 4) == STRIDE
    assert attend(n=4, blocks=FAKE + 2) == STRIDE
    # wider rows are taken, narrower ones are not
    t = dict(layout=TND, table=None)
    wide = desc((9, 2, 128), (768, 128, 1))
    assert attend(k=wide, v=wide, **t) == OK
    thin = desc((9, 2, 128), (128, 128, 1))
    assert attend(k=thin, v=wide, **t) == STRIDE


def test_attention_attributes():
    for mode in (1, 2, -1):
        assert attend(mode=mode) == ATTR
    for scale in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert attend(scale=scale) == ATTR
    for n in (65, -1):
        assert attend(n=n, blocks=FAKE) == ATTR


def test_attention_workspace():
    lib = m.load_library()
    need = m.msa_attention_workspace(2, 1, 8, 2, 1024)
    assert need > 0 and need % (2 * 8 * (128 * 4 + 8)) == 0
    k = desc((6, 128, 2, 128))
    args = dict(q=desc((2, 8, 128)), k=k, v=k, mb=1024)
    assert attend(**args) == WORKSPACE
    assert attend(ws=FAKE, wb=need - 1, **args) == WORKSPACE
    assert attend(ws=None, wb=need, **args) == WORKSPACE
    assert m.msa_attention_workspace(2, 1, 8, 2, 1024, 1) == 0     # one block is not split
    assert m.msa_attention_workspace(0, 1, 8, 2, 1024) == 0
    for bad in ((2, 0, 8, 2, 4), (2, 1, 8, 3, 4), (2, 1, 0, 2, 4), (2, 1, 8, 2, -1)):
        assert m.msa_attention_workspace(*bad) == 0
    assert lib.msa_status_str(WORKSPACE) != lib.msa_status_str(99)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------


def dims(shape, stride=None, dtype=F16, addr=FAKE):
    d = desc(shape, stride, dtype, addr)
    return (d.data or 0, d.dtype, d.ndim, *d.shape, *d.stride)


SRC = dims((0, 2, 128))
DST = dims((6, 128, 2, 128))


def item(src=SRC, dst=DST, scale=0, layout=BBND, rotate=1):
    return ITEM.pack(*src, *dst, scale, layout, rotate)


def append(*items, cos=FAKE, sin=FAKE, pos=64, rot=128, pairs=0, table=FAKE, mb=4, cu=FAKE,
           kv=FAKE, B=1, bs=128, n=None, null=False):
    buf = ctypes.create_string_buffer(b"".join(items) or b"\0" * ITEM.size)
    return m.load_library().msa_cache_append(
        None if null else ctypes.addressof(buf), len(items) if n is None else n, cos, sin, pos,
        rot, pairs, table, mb, cu, kv, B, bs, None)


def test_append_valid_empty_calls():
    assert append(item()) == OK
    assert append(*[item()] * 8) == OK
    assert append(item(rotate=0), cos=None, sin=None, pos=0, rot=0) == OK
    assert append(item(dst=dims((0, 2, 128)), layout=ROWS), table=None, mb=0) == OK
    assert append(item(dst=dims((0, 2, 128), addr=0), layout=TND), table=None, mb=0) == OK
    assert append(item(src=dims((0, 1, 128)), dst=dims((6, 128, 64), dtype=MX))) == OK


def test_append_rejects():
    assert append(null=True, n=1) == NULL
    assert append(item(), cu=None) == NULL
    assert append(item(), kv=None) == NULL
    assert append(item(), table=None) == NULL
    assert append(n=0) == ATTR
    assert append(*[item()] * 9) == ATTR
    assert append(item(rotate=2)) == ATTR
    for rot in (0, 8, 24, 144, -16):
        assert append(item(), rot=rot) == ATTR, rot
    assert append(item(), pairs=2) == ATTR
    assert append(item(), pos=-1) == SHAPE
    assert append(item(), bs=64) == SHAPE
    assert append(item(), mb=0) == SHAPE
    assert append(item(layout=4)) == LAYOUT
    assert append(item(layout=-1)) == LAYOUT
    assert append(item(), cos=FAKE + 4) == STRIDE
    assert append(item(), sin=FAKE + 8) == STRIDE


def test_append_types_and_scales():
    assert append(item(dst=dims((6, 128, 2, 128), dtype=BF16))) == DTYPE
    assert append(item(src=dims((0, 2, 128), dtype=E4M3))) == DTYPE
    assert append(item(dst=dims((6, 128, 2, 128), dtype=7))) == DTYPE
    assert append(item(), item(src=dims((0, 2, 128), dtype=BF16),
                               dst=dims((6, 128, 2, 128), dtype=BF16))) == DTYPE
    src = dims((2, 2, 128))
    assert append(item(src=src, dst=dims((6, 128, 2, 128), dtype=I8))) == SCALE
    assert append(item(src=src, dst=dims((6, 128, 2, 64), dtype=MX))) == SCALE
    assert append(item(src=src, scale=FAKE)) == SCALE
    assert append(item(src=src, dst=dims((6, 128, 2, 128), dtype=E5M2), scale=FAKE)) == SCALE
    assert append(item(src=src, dst=dims((6, 128, 2, 128), dtype=I8), scale=FAKE + 2)) == STRIDE


def test_append_shapes_and_strides():
    for src in ((0, 2, 64), (0, 3, 128), (0, 2), (0, 0, 128)):
        assert append(item(src=dims(src))) == SHAPE, src
    for dst in ((6, 128, 1, 128), (6, 64, 2, 128), (6, 128, 2, 64), (0, 128, 2, 128)):
        assert append(item(dst=dims(dst))) == SHAPE, dst
    assert append(item(dst=dims((6, 128, 2, 128), dtype=MX))) == SHAPE
    assert append(item(), item(src=dims((1, 2, 128)))) == SHAPE
    two = dims((2, 2, 128))
    assert append(item(src=two, dst=dims((3, 2, 128)), layout=ROWS)) == SHAPE
    assert append(item(src=dims((2, 2, 128), (256, 128, 2)))) == STRIDE
    assert append(item(src=dims((2, 2, 128), (260, 128, 1)))) == STRIDE
    assert append(item(src=dims((2, 2, 128), (256, 132, 1)))) == STRIDE
    assert append(item(src=dims((2, 2, 128), (-256, 128, 1)))) == STRIDE
    assert append(item(src=dims((0, 2, 128), addr=FAKE + 2))) == STRIDE
    assert append(item(dst=dims((6, 128, 2, 128), (32768, 256, 136, 1)))) == STRIDE
    # rows that overlap would be written by two waves
    assert append(item(src=two, dst=dims((2, 2, 128), (0, 128, 1)), layout=ROWS)) == STRIDE
    assert append(item(src=two, dst=dims((2, 2, 128), (256, 0, 1)), layout=ROWS)) == STRIDE
    assert append(item(src=two, dst=dims((9, 2, 128), (512, 128, 1)), layout=TND),
                  table=None, mb=0) == STRIDE
    # a token's heads between another token's heads; heads outside tokens are taken
    assert append(item(src=two, dst=dims((2, 2, 128), (128, 128, 1)), layout=ROWS)) == STRIDE
    three = dims((3, 2, 128))
    assert append(item(src=three, dst=dims((3, 2, 128), (128, 256, 1)), layout=ROWS)) == STRIDE
    assert append(item(src=three, dst=dims((3, 2, 128), (128, 384, 1), addr=0),
                       layout=ROWS)) == NULL
    # pages that overlap
    assert append(item(src=two, dst=dims((6, 128, 2, 128), (32752, 256, 128, 1)))) == STRIDE
    assert append(item(src=dims((2, 2, 128), addr=0))) == NULL
    assert append(item(src=two), cos=None) == NULL


# ---------------------------------------------------------------------------
# the binding's own checks (sizes that the C ABI takes on trust)
# ---------------------------------------------------------------------------


def args(T=2, B=2, MB=4, **kw):
    a = dict(query=torch.zeros(T, 8, 128, dtype=torch.float16),
             key=torch.zeros(6, 128, 2, 128, dtype=torch.float16),
             value=torch.zeros(6, 128, 2, 128, dtype=torch.float16),
             block_table=torch.zeros(B, MB, dtype=torch.int32),
             cu_seqlens_q=torch.zeros(B + 1, dtype=torch.int32),
             kv_len=torch.zeros(B, dtype=torch.int32), layout="BBND", sparse_mode=3,
             softmax_scale=None, out=torch.zeros(T, 8, 128, dtype=torch.float16), max_blocks=MB,
             stream=0)
    return a | kw


@pytest.mark.parametrize("change", [
    dict(cu_seqlens_q=torch.zeros(2, dtype=torch.int32)),
    dict(kv_len=torch.zeros(2, 1, dtype=torch.int32)),
    dict(kv_len=torch.zeros(2, dtype=torch.int64)),
    dict(block_table=torch.zeros(1, 4, dtype=torch.int32)),
    dict(block_table=torch.zeros(2, 5, dtype=torch.int32)),
    dict(block_table=torch.zeros(4, 2, dtype=torch.int32).t()),
    dict(block_table=None),
    dict(out=torch.zeros(2, 8, 64, dtype=torch.float16)),
    dict(out=torch.zeros(2, 8, 128)),
    dict(out=torch.zeros(2, 128, 8, dtype=torch.float16).transpose(1, 2)),
    dict(lse=torch.zeros(8, 2)),
    dict(lse=torch.zeros(2, 8, dtype=torch.float64)),
    dict(query=torch.zeros(16, 128, dtype=torch.float16)),
    dict(workspace=torch.zeros(8, 8).t()[1:]),
])
def test_binding_rejects(change):
    with pytest.raises(ValueError):
        m.msa_attention(**args(**change))


def test_binding_accepts_t0_and_checks_blocks():
    empty = dict(T=0)
    m.msa_attention(**args(**empty))
    a = args(**empty)
    m.msa_block_attention(blocks=torch.zeros(0, 2, 4, dtype=torch.int32), **a)
    for bad in (torch.zeros(0, 8, 4, dtype=torch.int32), torch.zeros(0, 2, 4),
                torch.zeros(0, 2, dtype=torch.int32), torch.zeros(1, 2, 4, dtype=torch.int32)):
        with pytest.raises(ValueError):
            m.msa_block_attention(blocks=bad, **a)
    with pytest.raises(ValueError):
        m.msa_block_attention(blocks=None, **a)
    with pytest.raises(m.MsaLayoutError):
        m.msa_attention(**args(T=0, layout="ROWS"))


def app(T=0, B=2, MB=4, **kw):
    a = dict(items=[m.CacheItem(torch.zeros(T, 2, 128, dtype=torch.float16),
                                torch.zeros(6, 128, 2, 128, dtype=torch.float16), "BBND",
                                rotate=True)],
             cos=torch.zeros(9, 64), sin=torch.zeros(9, 64),
             block_table=torch.zeros(B, MB, dtype=torch.int32),
             cu_seqlens_q=torch.zeros(B + 1, dtype=torch.int32),
             kv_len=torch.zeros(B, dtype=torch.int32), stream=0)
    return a | kw


def test_append_binding():
    m.msa_cache_append(**app())
    src = torch.zeros(0, 1, 128, dtype=torch.float16)
    i8 = torch.zeros(6, 128, 1, 128, dtype=torch.int8)
    good = m.CacheItem(src, i8, "bbnd", scale=torch.zeros(6, 1, 128))
    m.msa_cache_append(**app(items=[good]))
    for scale in (torch.zeros(6, 1, 64), torch.zeros(6, 1, 128, dtype=torch.float64),
                  torch.zeros(6, 128, 2)[:, :, 0]):
        with pytest.raises(ValueError):
            m.msa_cache_append(**app(items=[good._replace(scale=scale)]))
    for change in (dict(items=[]), dict(items=[good] * 9), dict(cos=None),
                   dict(cos=torch.zeros(9, 32)), dict(sin=torch.zeros(9, 64).double()),
                   dict(cos=None, sin=None), dict(block_table=None),
                   dict(cu_seqlens_q=torch.zeros(2, dtype=torch.int32)),
                   dict(kv_len=torch.zeros(2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            m.msa_cache_append(**app(**change))
    with pytest.raises(m.MsaError):
        m.msa_cache_append(**app(items=[good._replace(layout="XYZ")]))
    with pytest.raises(m.MsaError):
        m.msa_cache_append(**app(cos=torch.zeros(9, 4), sin=torch.zeros(9, 4)))


def test_binding_refuses_host_tensors():
    # well-formed, but the kernels would be given addresses of host memory
    for a in (args(), args(query=torch.zeros(2, 8, 128, dtype=torch.float16))):
        with pytest.raises(ValueError, match="on a GPU"):
            m.msa_attention(**a)
    with pytest.raises(ValueError, match="on a GPU"):
        m.msa_block_attention(blocks=torch.zeros(2, 2, 4, dtype=torch.int32), **args())
    with pytest.raises(ValueError, match="on a GPU"):
        m.msa_cache_append(**app(T=2))


def test_launches_hold_less_than_2_32_threads():
    # 2^31 - 1 tokens of 16 heads would need 2^37 workgroups' threads
    T = 2**31 - 1
    assert attend(q=desc((T, 16, 128)), T=T) == SHAPE
    assert attend(q=desc((T, 16, 128)), n=16, blocks=FAKE, T=T) == SHAPE
    one = dict(layout=ROWS, rotate=0)
    assert append(item(src=dims((T, 2, 128)), dst=dims((T, 2, 128)), **one), table=None,
                  mb=0) == SHAPE


def test_allocating_forms_reject():
    a = args(T=0)
    rest = (a["key"], a["value"], a["block_table"], a["cu_seqlens_q"], a["kv_len"], "BBND")
    for q in (torch.zeros(16, 128, dtype=torch.float16), torch.zeros(128, dtype=torch.float16)):
        with pytest.raises(ValueError):
            m.attention(q, *rest)
        with pytest.raises(ValueError):
            m.block_attention(q, *rest[:2], torch.zeros(0, 2, 4, dtype=torch.int32), *rest[2:])
    with pytest.raises(ValueError):
        m.block_attention(a["query"], *rest[:2], None, *rest[2:])
