"""Prompt attention where bits must not change: what a row does not see, and bad offsets elsewhere."""
import numpy as np
import pytest

import workloads as wl
from tests.test_kv_gpu import mbd  # noqa: F401  (mbd is the fixture)
from tests.test_prompt_gpu import NAN, check, make, run

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


def test_rows_of_mostly_empty_sequences(mbd):
    """Sixteen million sequences, nearly all of them empty, and 64 pairs of heads: each CTA goes through seven million indexes
    that are no tile's, which takes longer than a wait's limit, while its other warps wait."""
    n, hq, hkv, d = 1 << 24, 128, 1, 64
    rng = np.random.default_rng(3)
    lens = np.zeros(n, np.int64)
    at = [0, 1, 31, 32, 1000, n // 2, n - 33, n - 2, n - 1]
    lens[at] = [1, 40, 3, 129, 2, 300, 5, 1, 130]
    qkv, cu = make(rng, lens, hq, hkv, d, pad=30)
    mbd.device_error_flags(clear=True)
    out, lse = run(mbd, qkv, cu, hq, hkv, d, 0.1)
    assert mbd.device_error_flags() == 0
    some = np.concatenate([[0], np.cumsum(lens[at])]).astype(np.int32)
    want, want_lse = run(mbd, qkv, some, hq, hkv, d, 0.1)
    np.testing.assert_array_equal(out, want)
    np.testing.assert_array_equal(lse, want_lse)


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 2), (64, 3, 3), (64, 2, 1), (256, 2, 1), (128, 1, 1)])
@pytest.mark.parametrize("window", [0, 1, 70, 200])
def test_prefixes(mbd, d, hq, hkv, window):
    """A prompt's first rows have the bits that they have without the rest of it, and with another rest."""
    rng = np.random.default_rng(d + window)
    qkv, cu = make(rng, [420], hq, hkv, d, sigma=3.0)
    # logits whose maximum moves: late queries meet the keys of every block with growing size
    qkv[:, :hq * d] = np.where(rng.random((420, 1)) < 0.2, qkv[:, :hq * d] + 0x100, qkv[:, :hq * d])   # (four times as large)
    whole, whole_lse = run(mbd, qkv, cu, hq, hkv, d, d ** -0.5, window)
    for length in (1, 2, 17, 33, 100, 127, 128, 129, 200, 255, 257, 300, 385):
        cut, cut_lse = run(mbd, np.ascontiguousarray(qkv[:length]), np.array([0, length], np.int32), hq, hkv, d, d ** -0.5, window)
        np.testing.assert_array_equal(cut, whole[:length], f"{length}")
        np.testing.assert_array_equal(cut_lse, whole_lse[:length], f"{length}")
        other = qkv.copy()
        other[length:] = make(rng, [420 - length], hq, hkv, d, sigma=20.0)[0]
        out, lse = run(mbd, other, cu, hq, hkv, d, d ** -0.5, window)
        np.testing.assert_array_equal(out[:length], whole[:length], f"{length}")
        np.testing.assert_array_equal(lse[:length], whole_lse[:length], f"{length}")


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 2), (64, 3, 3), (64, 2, 1), (256, 2, 1), (128, 1, 1)])
@pytest.mark.parametrize("window", [0, 1, 50, 128, 200])
def test_masked_values_change_no_bit(mbd, d, hq, hkv, window):
    """NaN and infinite rows after a row and before its window: the bits are those of a prompt where they are finite. Rows that see
    an infinite value alone have it, beside the finite columns' bits."""
    rng = np.random.default_rng(d + window)
    length = 520
    qkv, cu = make(rng, [150, length], hq, hkv, d, pad=20, sigma=0.5)
    base, base_lse = run(mbd, qkv, cu, hq, hkv, d, 0.02, window)
    kv = slice(hq * d, (hq + 2 * hkv) * d)
    v0 = (hq + hkv) * d
    for at in (0, 1, 100, 127, 128, 200, 255, 256, 300, 383, 384, 519):
        row = int(cu[1]) + at
        sees = np.zeros(len(qkv), bool)
        sees[row:min(cu[2], row + window) if window else cu[2]] = True
        odd = qkv.copy()
        odd[row, kv] = rng.choice([NAN, 0x7F80, 0xFF80], odd[0, kv].shape)
        odd[row, :hq * d] = NAN
        out, lse = run(mbd, odd, cu, hq, hkv, d, 0.02, window)
        keep = ~sees
        keep[cu[-1]:] = False
        np.testing.assert_array_equal(out[keep], base[keep], f"{at}")
        np.testing.assert_array_equal(lse[keep], base_lse[keep], f"{at}")
        one = qkv.copy()                             # an infinite value alone: of the last key-value head, in one column
        one[row, v0 + hkv * d - 3] = 0xFF80
        out, lse = run(mbd, one, cu, hq, hkv, d, 0.02, window)
        want = base.copy()
        want[sees, (hkv - 1) * (hq // hkv):, d - 3] = 0xFF80
        want[cu[-1]:] = 0x5A5A
        np.testing.assert_array_equal(out, want, f"{at}")
        np.testing.assert_array_equal(lse, base_lse)


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 2), (64, 3, 3), (256, 1, 1)])
@pytest.mark.parametrize("rise", [4.0, 5.5, 5.6, 10.9, 11.3, 40.0])   # of the logits, from each block to the next: 2^8 is 5.55
def test_large_values_under_rising_logits(mbd, d, hq, hkv, rise):
    """Sums stay in range for the values that the header allows (2^8 times 700 keys times 2^102 is below 2^120), whether the maximum
    that they are relative to is kept from block to block or not."""
    rng = np.random.default_rng(d)
    qkv, cu = make(rng, [700], hq, hkv, d)
    k0, v0 = hq * d, (hq + hkv) * d
    qkv[:, :k0] = wl.f32_to_bf16_bits(np.full((700, hq * d), 0.5, np.float32))
    qkv[:, k0:v0] = wl.f32_to_bf16_bits(np.repeat(np.arange(700, dtype=np.float32)[:, None] // 128 * (rise / d * 20), hkv * d, 1))
    qkv[:, v0:v0 + hkv * d] += 100 << 7
    check(mbd, qkv, cu, hq, hkv, d, scale=0.1)
