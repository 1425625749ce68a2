"""Where the binding's outputs and workspaces come from: torch's ordinary allocation, which
dispatch modes see and deterministic mode fills."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from moe_grouped_gemm_wgrad_gb300 import mgw

pytestmark = pytest.mark.gpu


def _inputs():
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(256, 128, generator=g, device="cuda").bfloat16()
    off = torch.tensor([0, 100, 256], dtype=torch.int32, device="cuda")
    logits = torch.randn(64, 16, generator=g, device="cuda")
    return x, off, logits


def test_allocations_are_seen_by_dispatch_modes():
    x, off, logits = _inputs()

    class Seen(TorchDispatchMode):
        def __init__(self):
            super().__init__()
            self.shapes = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            r = func(*args, **(kwargs or {}))
            if "empty" in str(func):
                self.shapes.append(tuple(r.shape))
            return r

    with Seen() as seen:
        idx, w = mgw.moe_route(logits, 4)
        q, sc = mgw.mxfp8_quantize(x, off)
    assert seen.shapes == [(64, 4), (64, 4), tuple(q.shape), tuple(sc.shape)]


def test_deterministic_mode_fills_what_a_call_leaves_unwritten():
    """Rows of dy that no pair names are not written: torch.empty's fill shows in them."""
    before = torch.are_deterministic_algorithms_enabled()
    row_of = torch.tensor([[0, 2]], dtype=torch.int32, device="cuda")
    y, dout, w = torch.ones(4, 8, device="cuda"), torch.ones(1, 8, device="cuda"), torch.ones(1, 2, device="cuda")
    torch.use_deterministic_algorithms(True)
    try:
        dy, _ = mgw.moe_combine_backward(dout, y, row_of, weights=w)
    finally:
        torch.use_deterministic_algorithms(before)
    assert (dy[[0, 2]] == 1).all() and torch.isnan(dy[[1, 3]]).all()


# ------------------------------------------------------- calls on another stream than the current one
def _hold(stream):
    """A queue of some 100 ms on ``stream``."""
    with torch.cuda.stream(stream):
        m = torch.ones(8192, 8192, device="cuda")
        for _ in range(12):
            m = torch.mm(m, m).mul_(1.0 / 8192)
    return m


def _dispatch_inputs():
    g = torch.Generator(device="cuda").manual_seed(6)
    idx = torch.randint(0, 32, (20000, 8), generator=g, device="cuda", dtype=torch.int32)
    return idx, int(mgw.load().mgw_moe_dispatch_workspace_bytes(20000, 8, 32))


def test_dropped_tensors_are_kept_from_the_current_stream_until_the_call_is_done():
    idx, need = _dispatch_inputs()
    want = mgw.moe_dispatch(idx, 32)
    side = torch.cuda.Stream()
    # what the allocator does with a dropped tensor that nobody else uses: the same address again
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    at = ws.data_ptr()
    del ws
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() == at
    own = idx.clone()
    own_at = own.data_ptr()
    torch.cuda.synchronize()
    held = _hold(side)
    got = mgw.moe_dispatch(own, 32, workspace=ws, stream=side)
    side_at = [t.data_ptr() for t in mgw.moe_dispatch(own, 32, stream=side)]   # dropped at once
    del ws, own
    new = [torch.full((need,), 7, dtype=torch.uint8, device="cuda"), torch.full_like(idx, 7)]
    new += [torch.full_like(t, 7) for t in want]
    assert not side.query(), "the side stream was not held long enough for this test"
    assert not {t.data_ptr() for t in new} & {at, own_at, *side_at}
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((held > 0).all())


def test_a_call_on_another_stream_takes_no_memory_that_the_current_one_still_reads():
    g = torch.Generator(device="cuda").manual_seed(7)
    y = torch.randn(1024, 512, generator=g, device="cuda")
    row_of = torch.randperm(1024, generator=g, device="cuda").int().view(512, 2)
    want = mgw.moe_combine(y, row_of)
    side = torch.cuda.Stream()
    x = torch.randn(512, 512, generator=g, device="cuda")   # the size of the call's output
    kept, at = x.clone(), x.data_ptr()
    torch.cuda.synchronize()
    held = _hold(torch.cuda.current_stream())
    read = x * 1.0          # queued behind the work above
    del x                   # the host lets go of it before it is read
    out = mgw.moe_combine(y, row_of, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query(), "the current stream was not held long enough"
    assert out.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(read, kept) and bool((held > 0).all())


def test_a_result_outlives_its_reader_on_the_current_stream():
    """A result of a side stream's pool, read on the current stream and dropped, is not handed out to
    the side stream's next call before it has been read."""
    g = torch.Generator(device="cuda").manual_seed(8)
    y = torch.randn(1024, 512, generator=g, device="cuda")
    row_of = torch.randperm(1024, generator=g, device="cuda").int().view(512, 2)
    one_slot = row_of[:, :1].contiguous()
    want = mgw.moe_combine(y, row_of)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = mgw.moe_combine(y, row_of, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    held = _hold(torch.cuda.current_stream())
    read = out * 1.0
    at = out.data_ptr()
    del out
    other = mgw.moe_combine(y, one_slot, stream=side)
    assert other.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(read, want) and bool((held > 0).all())
