"""The Python binding's choice of stream, without a GPU."""
import types

import torch

import token_routing_expert_router_gb300 as moe


def test_current_stream_without_the_raw_call(monkeypatch):
    """torch's raw-handle call is a private one: a torch without it gives the public stream's handle."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=123))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert moe._stream() == 123
    assert moe._stream(types.SimpleNamespace(cuda_stream=7)) == 7


def test_current_stream_by_the_raw_call(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 40 + device, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
    assert moe._stream() == 42
