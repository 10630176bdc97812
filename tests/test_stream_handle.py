"""The binding's default stream: the current one's handle, by the short way where PyTorch has it, else by the public one."""
import types

import sparse_attention_dsa_gb300._lib as lib


def test_the_handle_of_the_current_stream(monkeypatch):
    cuda = types.SimpleNamespace(current_device=lambda: 3, current_stream=lambda: types.SimpleNamespace(cuda_stream=77))
    short = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda device: 1000 + device)
    monkeypatch.setattr(lib, "_torch", types.SimpleNamespace(cuda=cuda, _C=short))
    assert lib._stream(None) == 1003
    monkeypatch.setattr(lib, "_torch", types.SimpleNamespace(cuda=cuda, _C=types.SimpleNamespace()))
    assert lib._stream(None) == 77
    assert lib._stream(5) == 5
    assert lib._stream(types.SimpleNamespace(cuda_stream=9)) == 9
