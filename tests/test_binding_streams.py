"""The binding's streams, on CPU: which handle a call gets, with stand-ins for torch's queries."""
import types

import torch

from moe_grouped_gemm_wgrad_gb300 import mgw


def test_the_current_streams_handle_with_and_without_the_raw_query(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *d: types.SimpleNamespace(cuda_stream=0x50))
    monkeypatch.setattr(mgw, "_raw_stream", lambda device: 0x100 + device)
    assert mgw._stream(None) == 0x103
    assert mgw._stream(types.SimpleNamespace(cuda_stream=0x77)) == 0x77
    monkeypatch.setattr(mgw, "_raw_stream", None)
    assert mgw._stream(None) == 0x50


def test_the_device_of_a_call_is_made_current_only_when_it_is_not(monkeypatch):
    made = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", lambda d: made.append(d) or mgw._SAME_DEVICE)
    mgw._device(torch.device("cuda", 1))
    assert made == []
    mgw._device(torch.device("cuda", 0))
    assert made == [torch.device("cuda", 0)]
