"""Host-side checks of what a call of the key-value cache may overlap and how far its pools may reach (no GPU: each
fails before any CUDA call)."""
import pytest

import memory_bound_decoder_gb300 as mbd
from tests.test_kv_abi import CALLS, A, _rc, append, attend, cache, lib  # noqa: F401  (lib is the fixture)


@pytest.mark.parametrize("result", ["out", "lse", "workspace"])
@pytest.mark.parametrize("array,accumulate", [("weight", False), ("weight", True), ("position", False), ("position", True)])
def test_attention_results_apart_from_the_cache(lib, result, array, accumulate):
    """Results over the accumulated weights or the positions would destroy what the next eviction reads."""
    at = {"weight": 5 * A, "position": 6 * A}[array] + 256
    assert _rc(attend(cache(), accumulate=accumulate, **{result: at})) == mbd.ERR_INVALID_ARG


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stride", [0, 1 << 37])
def test_pools_beyond_every_range(lib, call, stride):
    """Dense pages whose pool would pass 2^64 bytes, where the ranges of the overlap checks wrap: refused, as with the
    stride given."""
    c = cache(n_pages=(1 << 31) - 1, page_size=65536, n_kv_heads=4096, head_dim=256, page_stride=stride, k=A, v=A)
    kw = dict(n_q_heads=4096) if call is attend else {}
    assert _rc(call(c, pages_per_seq=1, **kw)) == mbd.ERR_UNSUPPORTED


def test_pools_of_the_largest_extent(lib):
    """64 T elements, pages dense: taken (the call fails on its missing rows only)."""
    c = cache(n_pages=1 << 20, page_size=65536, n_kv_heads=4, head_dim=256)
    assert _rc(append(c, k=None, pages_per_seq=1)) == mbd.ERR_INVALID_ARG
