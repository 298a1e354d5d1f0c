"""The append to an NVFP4 cache of rows that hold NaN and infinities, byte for byte against the reference, and the attention over them."""
import numpy as np
import pytest

import workloads as wl
from tests.test_kv_gpu import bits, mbd, run_attend, up  # noqa: F401  (mbd is the fixture)
from tests.test_kv_nvfp4_gpu import Cache

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nan", [0x7FC1, 0xFFC0, 0x7F81])
def test_append_of_values_that_are_not_finite(mbd, d, nan):
    """A block that holds a NaN, in either half of it, anywhere, or nothing else, has a NaN for its scale, and its codes are zeros; an
    infinity counts as more than the largest value that a block can hold. Other blocks are as they were."""
    rng = np.random.default_rng(d)
    hkv, n = 3, 40
    c = Cache(rng, [n], hkv, d, 16, spare=1)
    c.device(mbd)
    x = [bits(rng, n, hkv * d).reshape(n, hkv, d) for _ in range(2)]
    for t in range(n):
        for a in x:
            h, e = rng.integers(hkv), int(rng.integers(d))
            block = slice(e // 16 * 16, e // 16 * 16 + 16)
            if t % 4 == 0:
                a[t, h, e] = nan
            elif t % 4 == 1:
                a[t, h, block] = nan
            elif t % 4 == 2:
                a[t, h, e] = 0xFF80 if t % 8 == 2 else 0x7F80
            else:
                a[t, h, block] = rng.choice([0x7F80, 0xFF80], 16)
                if t % 8 == 3:
                    a[t, h, e] = nan
    mbd.kv_cache_append(c.c, up(x[0].reshape(n, -1)), up(x[1].reshape(n, -1)), 0, c.table_d, c.width, c.lens_d, 1, n,
                        up(np.array([0, n], np.int32)))
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        c.store(0, np.arange(n), x[0], x[1])
    c.check_equal("append")
    scales = c.blocks(c.k_raw)[c.table[0, 0], :, :16]
    assert (scales == 0x7F).any() and (scales == 0x7E).any()
    assert mbd.device_error_flags() == 0


@pytest.mark.parametrize("page", [1, 8, 16, 64])
def test_attention_sees_an_appended_nan(mbd, page):
    """A broken key makes its head's result NaN, a broken value its block's columns: neither turns into a plausible number."""
    rng = np.random.default_rng(page)
    hq, hkv, d, n = 8, 2, 128, 70
    c = Cache(rng, [n, 20], hkv, d, page)
    c.device(mbd)
    k, v = (bits(rng, n, hkv * d) for _ in range(2))
    k[33, 5] = 0x7FC0                                # of head 0
    v[50, d + 40] = 0x7FC0                           # of head 1, in block 2
    mbd.kv_cache_append(c.c, up(k), up(v), 0, c.table_d, c.width, c.lens_d, 2, n,
                        up(np.array([0, n, n], np.int32)))
    _, out, lse, _ = run_attend(mbd, c, rng, hq)
    out = wl.bf16_bits_to_f32(out).reshape(2, hq, d)
    assert np.isnan(out[0, :4]).all() and np.isnan(lse.reshape(2, hq)[0, :4]).all()
    assert np.isnan(out[0, 4:, 32:48]).all() and np.isfinite(lse.reshape(2, hq)[0, 4:]).all()
    out[0, :4] = out[0, 4:, 32:48] = 0
    assert np.isfinite(out).all()
