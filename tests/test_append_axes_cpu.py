"""The append with position axes on the CPU: malformed calls are rejected before
anything is launched (each fails or has T = 0), and the oracle's rotation by axes
on a row worked by hand."""
import math

import torch

import block_max_qk_amd as m
from oracle import layer
from test_layer_boundary_cpu import FAKE, ITEM

OK, NULL, LAYOUT, DTYPE, SHAPE, STRIDE, SCALE, ATTR = range(8)


def item(T=2, H=2, rotate=1):
    s = (T, H, 128, 0, H * 128, 128, 1, 0)
    return ITEM.pack(FAKE, 1, 3, *s, 2 * FAKE, 1, 3, *s, 0, 3, rotate)


def call(it=None, rot=32, ap=FAKE, axes=3, pairs=bytes([0, 1, 2, 0] * 4), cos=FAKE):
    return m.load_library().msa_cache_append_axes(
        item() if it is None else it, 1, cos, FAKE, 10, rot, 0, ap, axes, pairs, None, 0, FAKE,
        FAKE, 1, 128, None)


def test_rejected():
    for axes in (0, -1, 5):
        assert call(axes=axes) == ATTR
    assert call(pairs=None) == NULL
    assert call(ap=None) == NULL
    assert call(ap=FAKE + 2) == STRIDE
    assert call(axes=2) == ATTR                               # a pair of axis 2
    assert call(pairs=bytes([0] * 15 + [3])) == ATTR
    assert call(cos=None) == NULL
    assert call(rot=24) == ATTR


def test_empty_calls():
    assert call(it=item(T=0)) == OK
    assert call(it=item(T=0), ap=None) == OK
    assert call(it=item(T=0, rotate=0), pairs=None, ap=None) == OK    # nothing is rotated


def test_oracle_by_hand():
    """Pair 0 by axis 1, pair 1 by axis 0: a quarter and a half turn."""
    x = torch.zeros(1, 1, 128)
    x[0, 0, :4] = torch.tensor([1.0, 2.0, 3.0, 4.0])
    turn = torch.tensor([0.0, math.pi / 2, math.pi])
    cos, sin = (f(turn)[:, None].expand(3, 2) for f in (torch.cos, torch.sin))
    ap = torch.tensor([[2], [1]], dtype=torch.int32)
    _, _, rows, _, _ = layer.append([x, torch.zeros(1, 1, 128), "ROWS", None, True], cos, sin, None,
                                    [0, 1], [1], False, True, ap, [1, 0])
    want = torch.tensor([-3.0, -2.0, 1.0, -4.0], dtype=torch.float64)
    assert torch.allclose(rows[0, 0, :4], want, atol=1e-6)
    assert not rows[0, 0, 4:].any()
