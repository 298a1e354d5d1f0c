"""Host-side edges of the serving step: entry points and references (no GPU)."""
import ctypes

import numpy as np
import pytest

import memory_bound_decoder_gb300 as mbd
from memory_bound_decoder_gb300 import build as mbd_build
from oracle import kv_nvfp4


@pytest.fixture(scope="module")
def lib():
    mbd_build.build()
    return mbd.get_lib()


@pytest.mark.parametrize("kw", [dict(amplitude=1e39), dict(amplitude=3.4028236e38), dict(amplitude=1.7e308)])
def test_amplitudes_that_fp32_does_not_hold_are_refused(lib, kw):
    """rotary() takes the amplitude in fp32 and refuses an infinite one: the table that leads there is refused, and not written."""
    args = mbd.RotaryScaling(0, 0, 10000.0, 1.0, 0.0, 1.0, 4.0, 32.0, 1.0, kw["amplitude"], None)
    turns, amp = (ctypes.c_uint64 * 8)(*[7] * 8), ctypes.c_float(5.0)
    assert lib.mbd_rotary_table(turns, ctypes.byref(amp), 16, ctypes.byref(args)) == mbd.ERR_INVALID_ARG
    assert list(turns) == [7] * 8 and amp.value == 5.0
    with pytest.raises(mbd.MbdError):
        mbd.rotary_table(16, **kw)
    assert mbd.rotary_table(16, amplitude=float(np.finfo(np.float32).max))[1] == np.finfo(np.float32).max


def test_reference_of_blocks_that_are_not_finite():
    """The NVFP4 reference: a NaN anywhere makes the block's scale NaN and its codes zeros; an infinity saturates."""
    x = np.ones((4, 32), np.float32)
    x[0, 3] = x[1, 20] = np.nan
    x[2, 5], x[3] = -np.inf, np.inf
    with np.errstate(invalid="ignore"):
        codes, scale = kv_nvfp4.encode(x, 2.0 ** -9)
    assert scale[0, 0] == scale[1, 1] == 0x7F and scale[2, 0] == 0x7E and (scale[3] == 0x7E).all()
    assert not codes[0, :8].any() and not codes[1, 8:].any() and codes[0, 8:].any() and codes[1, :8].any()
    assert codes[2, 2] >> 4 == 15 and (codes[3] == 0x77).all()
