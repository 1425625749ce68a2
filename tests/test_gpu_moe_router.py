"""More of the router on the GPU: masked experts beside gradients that are not finite."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_wgrad_gb300 import mgw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [16, 60, 100, 263, 1000])
@pytest.mark.parametrize("score", [mgw.SCORE_SOFTMAX, mgw.SCORE_SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_masked_experts_get_no_gradient_from_an_infinite_one(E, score, renorm, bad):
    """dlogits of a masked expert is 0 whatever the other experts' gradients are, and a token's
    gradients stay its own."""
    rng = np.random.default_rng(E)
    x = np.float32(rng.standard_normal((9, E)))
    x[rng.random((9, E)) < 0.4] = -np.inf
    x[:, 3] = 1.0
    g = np.float32(rng.standard_normal((9, E)))
    g[4, 3] = bad                               # a live expert of token 4
    g[np.isinf(x)] = np.nan                     # masked entries are not used
    logits = torch.from_numpy(x).cuda()
    idx, w = mgw.moe_route(logits, 4, score=score, renorm=renorm)
    for dw in (torch.ones_like(w), None):
        d = mgw.moe_route_backward(logits, idx, dw, dscores=torch.from_numpy(g).cuda(), score=score, renorm=renorm)
        d = d.cpu().numpy()
        assert (d[np.isinf(x)] == 0).all()
        assert np.isfinite(np.delete(d, 4, axis=0)).all() and not np.isfinite(d[4, 3])
