"""The binding's streams, on CPU: which handle a call gets, where its new tensors come from and what is
recorded, with stand-ins for torch's streams and the library."""
import contextlib
import types

import pytest
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
    monkeypatch.setattr(torch.cuda, "device", lambda d: made.append(d) or contextlib.nullcontext())
    mgw._device(torch.device("cuda", 1))
    assert made == []
    mgw._device(torch.device("cuda", 0))
    assert made == [torch.device("cuda", 0)]


# ----------------------------------------------------- calls on another stream than the current one
class StandIn:
    """A library that notes its calls, and whose sizes are right."""

    def __init__(self):
        self.calls = []

    def mgw_mxfp8_token_capacity(self, M, E):
        return (M + 127 * E + 127) // 128 * 128

    def mgw_mxfp8_scale_bytes(self, C, Mcap):
        return C * Mcap // 32

    def mgw_moe_dispatch_workspace_bytes(self, T, K, E):
        return 64

    def mgw_grouped_act_backward_workspace_bytes(self, E, M, N):
        return 64

    def __getattr__(self, name):
        if not name.startswith("mgw_"):
            raise AttributeError(name)

        def call(*args):
            self.calls.append(name)
            return 0
        return call


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def f32(*s):
    return torch.zeros(s)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


OFF = torch.tensor([0, 32, 64], dtype=torch.int32)
# (the call, tensors given, tensors it allocates)
CALLS = {
    "mxfp8_quantize": (lambda **k: mgw.mxfp8_quantize(bf(64, 128), OFF, **k), 2, 2),
    "mxfp8_quantize_gather": (lambda **k: mgw.mxfp8_quantize_gather(bf(9, 128), i32(64), OFF, **k), 3, 2),
    "grouped_wgrad_mxfp8": (lambda **k: mgw.grouped_wgrad_mxfp8(u8(128, 384), u8(1536), u8(256, 384), u8(3072), OFF, 64, **k), 5, 1),
    "grouped_wgrad_mxfp8_balanced": (lambda **k: mgw.grouped_wgrad_mxfp8_balanced(
        u8(128, 384), u8(1536), u8(256, 384), u8(3072), OFF, 64, u8(64), **k), 6, 1),
    "grouped_wgrad_mxfp8_balanced_noalloc": (lambda **k: mgw.grouped_wgrad_mxfp8_balanced_noalloc(
        u8(128, 384), u8(1536), u8(256, 384), u8(3072), OFF, 64, **k), 5, 1),
    "grouped_dgrad_f32": (lambda **k: mgw.grouped_dgrad_f32(f32(64, 32), f32(2, 32, 256), OFF, **k), 3, 1),
    "mxfp8_quantize_rows": (lambda **k: mgw.mxfp8_quantize_rows(bf(9, 128), OFF, row_index=i32(64), **k), 3, 2),
    "grouped_fprop_mxfp8": (lambda **k: mgw.grouped_fprop_mxfp8(u8(384, 128), u8(1536), u8(512, 128), u8(2048), OFF, 64, 256, **k), 5, 1),
    "grouped_dgrad_mxfp8": (lambda **k: mgw.grouped_dgrad_mxfp8(u8(384, 128), u8(1536), u8(256, 384), u8(3072), OFF, 64, **k), 5, 1),
    "moe_route": (lambda **k: mgw.moe_route(bf(4, 16), 2, bias=f32(16), with_scores=True, **k), 2, 3),
    "moe_route_backward": (lambda **k: mgw.moe_route_backward(bf(4, 16), i32(4, 2), f32(4, 2), f32(4, 16), **k), 4, 1),
    "moe_dispatch": (lambda **k: mgw.moe_dispatch(i32(5, 2), 3, **k), 1, 4),
    "grouped_fprop_mxfp8_act": (lambda **k: mgw.grouped_fprop_mxfp8_act(
        u8(384, 128), u8(1536), u8(512, 128), u8(2048), OFF, 64, 256, mgw.ACT_GELU, bias=f32(2, 256),
        residual=bf(64, 256), save_preact=True, **k), 7, 2),
    "grouped_act_backward": (lambda **k: mgw.grouped_act_backward(bf(64, 256), bf(64, 256), OFF, mgw.ACT_GELU, with_dbias=True, **k), 3, 3),
    "moe_combine": (lambda **k: mgw.moe_combine(bf(10, 64), i32(5, 2), weights=f32(5, 2), residual=bf(5, 64), **k), 4, 1),
    "moe_combine_backward": (lambda **k: mgw.moe_combine_backward(bf(5, 64), bf(10, 64), i32(5, 2), weights=f32(5, 2), **k), 4, 2),
}


def test_every_call_that_takes_a_stream_is_here():
    import inspect

    takes = {n for n, f in vars(mgw).items() if inspect.isfunction(f) and not n.startswith("_")
             and "stream" in inspect.signature(f).parameters}
    assert takes == set(CALLS)


@pytest.fixture
def world(monkeypatch):
    """Which stream is current at each allocation and launch, and what is recorded where."""
    here, side = FakeStream(0x10), FakeStream(0x20)
    w = {"now": here, "here": here, "side": side, "allocated": [], "recorded": [], "lib": StandIn()}

    @contextlib.contextmanager
    def as_current(s):
        before, w["now"] = w["now"], s
        yield
        w["now"] = before

    def empty(*a, **k):
        t = real_empty(*a, **k)
        w["allocated"].append((id(t), w["now"]))
        w.setdefault("keep", []).append(t)
        return t

    real_empty = torch.empty
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", as_current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *d: w["now"])
    monkeypatch.setattr(mgw, "_raw_stream", None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: w["recorded"].append((id(t), s)))
    monkeypatch.setattr(mgw, "load", lambda: w["lib"])
    monkeypatch.setattr(mgw, "_device", lambda dev: contextlib.nullcontext())
    return w


@pytest.mark.parametrize("name", sorted(CALLS))
def test_what_a_call_on_another_stream_allocates_and_records(world, name):
    """New memory comes from the pool of the stream that the call runs on (the current one's may
    still be in use there), and every tensor of the call is recorded on both streams."""
    call, given, made = CALLS[name]
    call(stream=world["side"])
    assert world["lib"].calls == ["mgw_" + name] and world["now"] is world["here"]
    assert [s for _, s in world["allocated"]] == [world["side"]] * made
    for s in (world["here"], world["side"]):
        assert len({t for t, r in world["recorded"] if r is s}) == given + made


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("how", [None, "here"])
def test_a_call_on_the_current_stream_records_nothing(world, name, how):
    call, _, made = CALLS[name]
    call(stream=how and FakeStream(world["here"].cuda_stream))
    assert [s for _, s in world["allocated"]] == [world["here"]] * made and world["recorded"] == []


def test_any_object_with_a_stream_handle_will_do(world, monkeypatch):
    class Foreign:
        cuda_stream = 0x30

    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle))
    mgw.moe_combine(bf(10, 64), i32(5, 2), stream=Foreign())
    assert [s.cuda_stream for _, s in world["allocated"]] == [0x30]
