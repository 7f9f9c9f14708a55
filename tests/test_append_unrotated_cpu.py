"""The append with position axes where no item is rotated: the axes are not looked
at, in the binding as at the C entry (no new tokens: nothing is launched)."""
import pytest
import torch

import block_max_qk_amd as m


def call(rotate, axis_positions, pair_axes, cos=None):
    src, dst = torch.zeros(2, 0, 2, 128, dtype=torch.bfloat16)
    ints = torch.zeros(3, dtype=torch.int32)
    m.msa_cache_append([m.CacheItem(src, dst, "ROWS", None, rotate)], cos, cos, None, ints[:2],
                       ints[2:], stream=0, axis_positions=axis_positions, pair_axes=pair_axes)


AXES = torch.zeros(3, 0, dtype=torch.int32)
COS = torch.ones(10, 16)


def test_not_looked_at():
    for pairs in ([0, 1, 2, 0] * 8, bytes([0, 1]), None):
        for axes in (AXES, AXES.long(), None):
            for cos in (None, COS):
                call(False, axes, pairs, cos)


def test_looked_at():
    call(True, AXES, [0, 1, 2, 0] * 4, COS)
    for axes, pairs in ((AXES, [0, 1]), (AXES, None), (AXES.long(), [0] * 16), (None, [0] * 16)):
        with pytest.raises(ValueError):
            call(True, axes, pairs, COS)
