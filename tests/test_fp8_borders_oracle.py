"""The layer oracle's fp8 encoder next to the border between two codes, on the
CPU: a binary64 value falls on its own side, however near."""
import pytest
import torch

from oracle import layer


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.float8_e5m2])
def test_own_side_of_every_border(dtype):
    codes = torch.arange(127, dtype=torch.int32).to(torch.uint8)
    vals = codes.view(dtype).double()
    codes, vals = codes[torch.isfinite(vals)], vals[torch.isfinite(vals)]
    middle = (vals[1:] + vals[:-1]) / 2
    for sign in (1.0, -1.0):
        for shift, want in ((-1e-15, codes[:-1]), (1e-15, codes[1:]),
                            (0.0, codes[:-1] + (codes[:-1] & 1))):
            row = torch.zeros(128, dtype=torch.float64)
            row[:len(middle)] = sign * middle * (1 + shift)
            assert (row.float()[:len(middle)].double() == sign * middle).all()
            got = layer.encode_fp8(row, dtype).view(torch.uint8)[:len(middle)]
            assert torch.equal(got, want + (128 if sign < 0 else 0))
