"""Host-side checks of what a call of the key-value cache may overlap and how far its pools may reach (no GPU: each
fails before any CUDA call)."""
import pytest

import memory_bound_decoder_gb300 as mbd
from tests.test_kv_abi import A, _rc, attend, cache, lib  # noqa: F401  (lib is the fixture)


@pytest.mark.parametrize("result", ["out", "lse", "workspace"])
@pytest.mark.parametrize("array,accumulate", [("weight", False), ("weight", True), ("position", False), ("position", True)])
def test_attention_results_apart_from_the_cache(lib, result, array, accumulate):
    """Results over the accumulated weights or the positions would destroy what the next eviction reads."""
    at = {"weight": 5 * A, "position": 6 * A}[array] + 256
    assert _rc(attend(cache(), accumulate=accumulate, **{result: at})) == mbd.ERR_INVALID_ARG
