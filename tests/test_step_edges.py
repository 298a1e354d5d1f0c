"""Host-side edges of the serving step: entry points and references (no GPU)."""
import numpy as np

from oracle import kv_nvfp4


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
