"""The binding's way to the current stream's handle does not depend on a private
name of torch being there."""
import types

import torch

from block_max_qk_amd import _binding


def test_without_torchs_private_getter(monkeypatch):
    asked = []

    def current_stream(dev):
        asked.append(dev)
        return types.SimpleNamespace(cuda_stream=0x1234)

    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(_binding, "_current_raw", None)
    assert _binding._raw_stream(None, 3) == 0x1234 and asked == [3]


def test_with_it(monkeypatch):
    monkeypatch.setattr(_binding, "_current_raw", lambda index: 100 + index)
    assert _binding._raw_stream(None, 2) == 102
    assert _binding._raw_stream(77, 2) == 77
