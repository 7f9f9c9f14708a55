"""Which tiles the sizes choose, and that the cases that mean a kernel reach it."""
import pytest

import block_max_qk_amd as m
import tile_cases


@pytest.mark.parametrize("name", list(tile_cases.CASES))
def test_cases_of_256_rows(name):
    at = tile_cases.sizes(name)
    assert m.msa_attention_tile_rows(*at) == 256
    assert (m.msa_attention_workspace(*at) > 0) == tile_cases.CASES[name][-1]


def test_the_other_tiles():
    rows = m.msa_attention_tile_rows
    assert rows(64, 64, 64, 8, 63) == 16           # a decode batch
    assert rows(128, 64, 64, 8, 63) == 16          # two tokens each
    assert rows(192, 64, 64, 8, 63) == 128         # three
    assert rows(1000, 1, 64, 8, 7) == 256          # a prompt
    assert rows(500, 1, 64, 8, 7) == 128
    assert rows(64, 64, 32, 4, 256, 16) == 16      # selected blocks
    assert rows(4096, 1, 32, 4, 256, 16) == 128


def test_sizes_that_no_call_takes():
    for at in ((0, 1, 8, 2, 4), (2, 0, 8, 2, 4), (2, 1, 8, 3, 4), (2, 1, 0, 2, 4), (2, 1, 8, 2, -1),
               (2 ** 31, 1, 8, 2, 4), (2, 1, 8, 2, 1 << 25), (2, 1, 8, 2, 4, 65),
               (2, 1, 1 << 17, 1, 4), (2, (1 << 30) + 1, 8, 2, 4), (2, 1, 8, 2, 4, -1)):
        assert m.msa_attention_tile_rows(*at) == 0 and m.msa_attention_workspace(*at) == 0
