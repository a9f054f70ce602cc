"""The stream that the binding hands to the library (no GPU needed)."""
from __future__ import annotations

import types

import torch

from software_pipelined_loop_gb300 import gemmpipe


def test_current_stream_without_torchs_raw_handle(monkeypatch):
    # The raw handle comes from a private function of torch; without it, from the Stream object.
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=4321))
    assert gemmpipe._stream(None) == 4321


def test_current_stream_is_the_raw_handle_of_the_current_device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 7)
    assert gemmpipe._stream(None) == 1007


def test_given_streams():
    assert gemmpipe._stream(0) == 0 and gemmpipe._stream(99) == 99
    assert gemmpipe._stream(types.SimpleNamespace(cuda_stream=55)) == 55
