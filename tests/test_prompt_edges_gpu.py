"""Prompt attention where bits must not change: what a row does not see, and bad offsets elsewhere."""
import numpy as np
import pytest

from tests.test_kv_gpu import mbd  # noqa: F401  (mbd is the fixture)
from tests.test_prompt_gpu import make, run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [256, 300, 5000])
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 64), (3, 3, 64), (1, 1, 256)])
def test_bad_offsets_among_many(mbd, n, hq, hkv, d):
    """A bad offset leaves out the two sequences that it bounds, is flagged, and changes nothing for the others, whatever their
    number."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 5, n)
    lens[rng.integers(0, n, 3)] = [0, 130, 300]
    lens[[0, 9, 10, n // 2, n - 1]] = [3, 2, 2, 2, 2]
    lens[n // 2 - 1] = lens[n - 2] = 1
    qkv, cu = make(rng, lens, hq, hkv, d, pad=3)
    mbd.device_error_flags(clear=True)
    want, want_lse = run(mbd, qkv, cu, hq, hkv, d, 0.1)
    assert mbd.device_error_flags() == 0
    for at, value in ((10, 10 ** 9), (10, -10 ** 9), (n // 2, int(cu[-1]) + 10), (n - 1, -1), (0, -1), (n, int(cu[-1]) + 10),
                      (n, 0)):
        bad = cu.copy()
        bad[at] = value
        out, lse = run(mbd, qkv, bad, hq, hkv, d, 0.1)
        assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX
        left = np.zeros(len(qkv), bool)
        left[cu[-1]:] = left[cu[max(at - 1, 0)]:cu[min(at + 1, n)]] = True
        np.testing.assert_array_equal(out[~left], want[~left], f"{at} {value}")
        np.testing.assert_array_equal(lse[~left], want_lse[~left], f"{at} {value}")
        assert (out[left] == 0x5A5A).all()
