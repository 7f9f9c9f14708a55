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


def test_workspace():
    """Never less than the plain scores' and at most a part per 4 blocks; 0 for sizes
    that no call takes."""
    part = 50 * 32 * (128 * 4 + 8)
    assert m.msa_attention_workspace(50, 1, 32, 4, 24) == 3 * part
    assert m.msa_attention_ex_workspace(50, 1, 32, 4, 24) == 6 * part
    for T in (1, 7, 50, 300, 2000, 9000):
        for B in (1, 2, 9, 64):
            for Hq, Hkv in ((8, 1), (32, 4), (64, 8), (12, 12)):
                for mb in (1, 4, 9, 40, 130, 1000):
                    plain = m.msa_attention_workspace(T, B, Hq, Hkv, mb)
                    most = m.msa_attention_ex_workspace(T, B, Hq, Hkv, mb)
                    row = T * Hq * (128 * 4 + 8)
                    assert plain <= most <= max(plain, row * -(-mb // 4)) and most % row == 0
    assert m.msa_attention_ex_workspace(50, 1, 32, 5, 24) == 0
    assert m.msa_attention_ex_workspace(50, 0, 32, 4, 24) == 0
