"""What the binding asks of torch and of tensors (CPU, stand-ins for both)."""
import sys
import types

import numpy as np
import pytest

import memory_bound_decoder_gb300 as mbd


def fake_torch(initialized=True, **c):
    cuda = types.SimpleNamespace(is_initialized=lambda: initialized, current_device=lambda: 3,
                                 current_stream=lambda: types.SimpleNamespace(cuda_stream=0x77))
    return types.SimpleNamespace(cuda=cuda, _C=types.SimpleNamespace(**c))


@pytest.mark.parametrize("torch,want", [
    (fake_torch(_cuda_getCurrentRawStream=lambda device: 0x50 + device), 0x53),
    (fake_torch(), 0x77),                                 # a torch without the name that is not public
    (fake_torch(initialized=False), None), (None, None)])
def test_current_stream_by_public_names_alone(monkeypatch, torch, want):
    monkeypatch.setitem(sys.modules, "torch", torch)
    assert mbd._stream(None) == want
    assert mbd._stream(5) == 5 and mbd._stream(types.SimpleNamespace(cuda_stream=6)) == 6


def test_pointers_of_any_integer_type():
    """An array object may answer data_ptr() with an integer that is not Python's: ctypes takes that only as an int."""
    array = types.SimpleNamespace(data_ptr=lambda: np.uint64(1 << 24))
    assert type(mbd._ptr(array)) is int
    c = mbd.kv_cache(array, 2 << 24, 8, 16, 2, 64)
    assert c.k == 1 << 24
    with pytest.raises(mbd.MbdError):                     # reaches the library's checks (no rows)
        mbd.kv_cache_append(c, array, None, 0, array, 4, array, 3, 3, stream=0)
