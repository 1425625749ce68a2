"""Clipping refuses tables in which memory that it writes belongs to another tensor too; the norm, which only
reads, takes them."""
import pytest
import torch

from moe_grouped_gemm_wgrad_gb300 import mgw
from test_adapters_abi import fake  # noqa: F401 (a fixture: the binding on a stand-in library)


def parts(dtype, *spans):
    flat = torch.zeros(64, dtype=dtype)
    return [flat[lo:hi] for lo, hi in spans]


BAD = [[(0, 64), (8, 16)], [(8, 16), (0, 64)], [(0, 9), (8, 16)], [(0, 8), (30, 40), (7, 9)], [(5, 6), (5, 6)], [(0, 64), (0, 1)]]
GOOD = [[(0, 8), (8, 16)], [(8, 16), (0, 8), (16, 64)], [(0, 64), (8, 8)], [(3, 3), (3, 3)]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spans", BAD, ids=str)
def test_in_place(fake, spans, dtype):
    grads = parts(dtype, *spans)
    for given in (grads, mgw.GradTable(grads), mgw.GradTable(grads, out=grads)):
        for _ in range(2):
            with pytest.raises(mgw.MgwError, match="two tensors"):
                mgw.clip_grads(given, 1.0)
        assert fake.calls == []
    mgw.grad_norm(grads)
    # read only: into memory of its own
    mgw.clip_grads(mgw.GradTable(grads, out=[g.clone() for g in grads]), 1.0)
    assert len(fake.calls) == 2
    # written twice
    with pytest.raises(mgw.MgwError, match="two tensors"):
        mgw.clip_grads(mgw.GradTable([g.clone() for g in grads], out=grads), 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("spans", GOOD, ids=str)
def test_neighbours(fake, spans, dtype):
    grads = parts(dtype, *spans)
    mgw.clip_grads(grads, 1.0)
    mgw.clip_grads(mgw.GradTable(grads, out=grads), 1.0)
    mgw.clip_grads(mgw.GradTable(grads, out=parts(dtype, *spans)), 1.0)
    mgw.clip_grads(mgw.GradTable(grads, out=[grads[0]] + parts(dtype, *spans[1:])), 1.0)
    assert len(fake.calls) == 4


def test_outputs_on_other_gradients(fake):
    a, b, c = parts(torch.bfloat16, (0, 16), (16, 32), (8, 24))
    for grads, out in (([a, b], [b, a]), ([a, b], [a, c]), ([a], [c]), ([a, b], [torch.zeros_like(a), a])):
        with pytest.raises(mgw.MgwError, match="two tensors"):
            mgw.clip_grads(mgw.GradTable(grads, out=out), 1.0)
    assert fake.calls == []
