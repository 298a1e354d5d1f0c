"""What the binding asks of torch and of tensors (CPU, stand-ins for both)."""
import sys
import types

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
