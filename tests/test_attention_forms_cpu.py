"""The entry of the capped, biased and narrowed attention on the CPU: malformed
calls are rejected before anything is launched; valid ones have T = 0."""
import ctypes

import block_max_qk_amd as m
from test_layer_boundary_cpu import BF16, FAKE, desc

OK, NULL, LAYOUT, DTYPE, SHAPE, STRIDE, SCALE, ATTR, HIP, WORKSPACE = range(10)


def call(T=0, cap=0.0, slopes=None, visible=None, scale=0.1, ws=None, wb=0, B=1, mb=4, k=None):
    q = desc((T, 8, 128), dtype=BF16)
    k = desc((6, 128, 2, 128), dtype=BF16) if k is None else k
    return m.load_library().msa_attention_ex(
        ctypes.byref(q), ctypes.byref(k), ctypes.byref(k), FAKE, mb, FAKE, FAKE, B, 128, 1, 3,
        scale, cap, slopes, visible, FAKE, None, ws, wb, None)


def test_valid_empty_calls():
    assert call() == OK
    assert call(cap=30.0, slopes=FAKE, visible=FAKE) == OK


def test_rejected():
    for cap in (-0.5, float("nan"), float("inf"), 3e38):
        assert call(cap=cap) == ATTR, cap
    assert call(cap=1e-44) == ATTR                          # scale / cap has no float32
    assert call(cap=1e-38, scale=1e3) == ATTR
    assert call(scale=1e-45, slopes=FAKE) == ATTR
    assert call(scale=1e-45) == OK
    assert call(slopes=FAKE + 2) == STRIDE
    assert call(visible=FAKE + 4) == STRIDE
    assert call(k=desc((6, 128, 2, 128))) == DTYPE          # what msa_attention rejects
    assert call(scale=0.0, cap=1.0) == ATTR
    assert call(T=2, mb=1000, cap=30.0) == WORKSPACE
