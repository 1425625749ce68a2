"""Gradient norm and clipping where the factor's quotient is not a number though its terms are, and tables
whose tensors overlap."""
import math

import pytest
import torch

from moe_grouped_gemm_wgrad_gb300 import mgw

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan
# few chunks go through one cluster, more through a launch each for the norm and the clipping
SIZES = {"cluster": [1000, 7], "launches": [3000000, 70001, 5], "tables": [33] * 1030}


def clipped(grads, **kw):
    """Into other buffers, and in place: the same bits."""
    outs = [torch.full_like(t, 9.0) for t in grads]
    norm = mgw.clip_grads(mgw.GradTable(grads, out=outs), **kw)
    mine = [t.clone() for t in grads]
    again = mgw.clip_grads(mine, **kw)
    assert again.item() == norm.item() or (again.isnan() and norm.isnan())
    assert all(torch.equal(p.nan_to_num(7.0), q.nan_to_num(7.0)) and torch.equal(p.isnan(), q.isnan())
               for p, q in zip(mine, outs))
    return norm.item(), outs


@pytest.mark.parametrize("where", sorted(SIZES))
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_factors_of_infinities_and_zeros(where, kind):
    def some(value):
        return [torch.full((n,), value, dtype=kind, device="cuda") for n in SIZES[where]]

    # an infinite norm: 0, whatever the limit; the infinity itself times 0 is none
    bad = some(2.0)
    bad[-1][3] = INF
    for limit in (INF, 1.0, 0.0):
        norm, outs = clipped(bad, max_norm=limit)
        assert norm == INF and outs[-1][3].isnan()
        outs[-1][3] = 0.0
        assert not any(t.any() for t in outs)
    # no limit: as they were
    for eps in (0.0, 1e-6, INF):
        assert all((t == 2.0).all() for t in clipped(some(2.0), max_norm=INF, eps=eps)[1])
        assert not any(t.any() for t in clipped(some(0.0), max_norm=INF, eps=eps)[1])
    # a limit of 0
    for eps in (0.0, 1e-6, INF):
        for value in (0.0, 2.0):
            norm, outs = clipped(some(value), max_norm=0.0, eps=eps)
            assert (norm == 0) == (value == 0) and not any(t.any() for t in outs)
    # zeros without eps under an ordinary limit
    assert not any(t.any() for t in clipped(some(0.0), max_norm=1.0, eps=0.0)[1])
    # a norm that is not a number: all are none, whatever the limit
    bad[-1][3] = NAN
    for limit in (INF, 1.0, 0.0):
        norm, outs = clipped(bad, max_norm=limit)
        assert math.isnan(norm) and all(t.isnan().all() for t in outs)


@pytest.mark.parametrize("known,limit,factor", [(INF, INF, 0.0), (0.0, 0.0, 0.0), (0.0, 1.0, 1.0), (4.0, INF, 1.0),
                                                (NAN, INF, NAN), (NAN, 0.0, NAN), (4.0, 2.0, 0.5)])
def test_factors_of_a_known_norm(known, limit, factor):
    t = torch.full((1,), known, device="cuda")
    for n in (10, 3000000):
        g = torch.full((n,), 3.0, device="cuda")
        mgw.clip_grads([g], limit, known_norm=t, eps=0.0)
        assert g.isnan().all() if math.isnan(factor) else (g == 3.0 * factor).all()
