"""Host-side checks of a cache held in NVFP4 (no GPU) and pins of its NumPy reference."""
import numpy as np
import pytest

import memory_bound_decoder_gb300 as mbd
import workloads as wl
from oracle import kv_nvfp4 as ref
from tests.test_kv_abi import CALLS, A, _rc, append, attend, cache, lib  # noqa: F401  (lib is the fixture)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,status", [
    (dict(mode="dynamic"), mbd.ERR_INVALID_ARG), (dict(mode=2), mbd.ERR_INVALID_ARG),
    (dict(k_scale=None), mbd.ERR_INVALID_ARG), (dict(v_scale=None), mbd.ERR_INVALID_ARG),
    (dict(k_scale=A + 64), mbd.ERR_INVALID_ARG), (dict(k_scale=A + 2 * 16 * 32 + 16), mbd.ERR_INVALID_ARG),
    (dict(page_stride=2 * 16 * 36 - 16), mbd.ERR_INVALID_ARG), (dict(v=A + 2 * 16 * 36 * 8 - 16), mbd.ERR_INVALID_ARG),
    (dict(page_stride=2 * 16 * 36 + 8), mbd.ERR_MISALIGNED), (dict(v_scale=4 * A + 2), mbd.ERR_MISALIGNED),
    (dict(head_dim=80), mbd.ERR_UNSUPPORTED),
])
def test_descriptions(lib, call, kw, status):
    assert _rc(call(cache(fmt="nvfp4", **kw))) == status


def test_accepted(lib):
    """Pools side by side, interleaved pages, pages of one short row: only the missing rows are refused."""
    for kw in (dict(v=A + 2 * 16 * 36 * 8), dict(v=A + 1152, page_stride=2304), dict(n_kv_heads=1, page_size=1, v=A + 48 * 8)):
        assert _rc(append(cache(fmt="nvfp4", **kw), k=None)) == mbd.ERR_INVALID_ARG
        c = cache(fmt="nvfp4", **kw)
        assert mbd.paged_attention_workspace_bytes(c, 4, 3, 4, False) > 0
        mbd.kv_cache_append(c, None, None, 0, None, 4, None, 0, 0)
    c = cache(fmt="nvfp4", n_kv_heads=1, page_size=1, v=A + 48 * 8 - 16)   # dense pages are rounded up to 48 bytes
    assert _rc(attend(c, q=14 * A)) == mbd.ERR_INVALID_ARG


def test_reference_codes():
    x = np.array([0, 0.25, 0.2500001, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 5.0001, 7, -0.0, -0.25, -6])
    assert list(ref.E2M1[ref.e2m1_codes(x)]) == [0, 0, 0.5, 1, 1, 2, 2, 4, 4, 6, 6, 0, 0, -6]
    assert list(ref.e2m1_codes(x)[-3:-1]) == [8, 8]


def test_reference_rows():
    """The largest element of a block lands near 6 codes; what is stored comes back within half a step."""
    rng = np.random.default_rng(0)
    x = wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(rng.standard_normal((9, 64)).astype(np.float32))).astype(np.float64)
    codes, sf = ref.encode(x, 2.0 ** -9)
    assert codes.shape == (9, 32) and sf.shape == (9, 4)
    y = ref.decode(codes, sf, 2.0 ** -9)
    scale = (ref.base.E4M3[sf] * 2.0 ** -9).repeat(16, -1)
    steps = np.abs(x) / scale
    half = np.where(steps < 2, 0.25, np.where(steps < 4, 0.5, 1.0)) * scale
    assert (np.abs(x - y) <= half * (1 + 1e-12)).all() and (steps.reshape(9, 4, 16).max(-1) > 5.3).all()
