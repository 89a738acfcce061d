"""Sizes of the norm's calls whose product passes 64 bits: refused, not taken for a
call without rows (CPU: every call fails before the device is touched)."""
import ctypes

import pytest

FAKE = 1 << 20


@pytest.fixture(scope="module")
def abi():
    from long_context_linear_b200 import _abi
    return _abi


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("B,N,Hq,Hk", [
    (1 << 30, 1 << 30, 16, 0),           # B N H = 2^64
    (1 << 30, 1 << 30, 8, 8),
    (1 << 30, 1 << 30, 10, 6),
    (1 << 30, 1 << 30, 9, 0),            # negative as 64 bits
    ((1 << 31) - 1, 1 << 30, 1 << 20, 1 << 20),
    (1 << 20, 1 << 20, 1, 0), (1, 1 << 30, 1 << 20, 0), (1 << 14, 1 << 20, 1, 1),
    (1, (1 << 30) + 1, 1, 1), (1, 1, (1 << 20) + 1, 1), (1, 1, 1, (1 << 20) + 1),
])
def test_too_large(abi, B, N, Hq, Hk, backward):
    v = ctypes.byref(abi.View(FAKE, 1024, 1024, 1024))
    mid, tail = (FAKE, FAKE, FAKE, None, 0, 0, 0), (B, N, Hq, Hk, 128, 64, 1e-6, 0, 0, 0)
    if backward:
        st = abi.lib.la_qk_norm_rope_backward(v, v, v, v, *mid, v, v, FAKE, FAKE, *tail, FAKE, 1 << 30, None)
    else:
        st = abi.lib.la_qk_norm_rope(v, v, v, v, *mid, *tail, None)
    assert st == 1 and b"too large" in abi.lib.la_last_error()
