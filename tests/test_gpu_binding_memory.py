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
