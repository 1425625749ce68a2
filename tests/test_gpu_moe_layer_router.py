"""The router's gradient of the example layer against autograd in fp32, where it nearly cancels.

dlogit[e] = p[e] (dw[e] - sum_j p[j] dw[j]) with dw[e] = dout . y[e]: of few tokens the terms are nearly equal
numbers, so an error of y that is small beside y may be large beside the gradient.  The tolerance is therefore
relative to the terms before they cancel.  Two chained products of e4m3 operands are off by 5 to 8% of their rms
(as in test_gpu_moe_layer.py), by an independent rounding for each of y's H elements, so dw[e] is off by
0.08 |dout| |y[e]| / sqrt(H) as a standard deviation, and by six of them at most; the gradient's element [e, k] by the
sum over the tokens of

    6 0.08 H^-1/2 |x[k]| p[e] (|dout| |y[e]| + sum_j p[j] |dout| |y[j]|).

fp32's own roundings (H terms, 2^-24 each) are far below."""
import pytest
import torch

from test_gpu_moe_layer import moe_ffn  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def layer_and_autograd(moe_ffn, seed, tokens, hidden, ffn, experts, top_k):
    """-> (the layer's router gradient, autograd's, the bound), inputs from ``seed``."""
    with torch.random.fork_rng(devices=[0]):
        torch.manual_seed(seed)
        layer = moe_ffn.MoeFfn(hidden, ffn, experts, top_k, seed=tokens)
        layer.b1.normal_(std=0.3)
        layer.b2.normal_(std=0.3)
        x = torch.randn(tokens, hidden, device="cuda").bfloat16()
        dout = torch.randn(tokens, hidden, device="cuda").bfloat16()
    layer.forward(x)
    got = layer.backward(dout)[1]["router"]
    idx = layer.saved[2].long()
    p = {k: v.clone().requires_grad_() for k, v in layer.parameters().items()}
    xr = x.float()
    w = torch.softmax((xr @ p["router"].t()).gather(1, idx), 1)
    ys = torch.zeros(tokens, top_k, hidden, device="cuda")
    for e in range(experts):
        t, k = (idx == e).nonzero(as_tuple=True)
        if t.numel():
            z = xr[t] @ p["w1"][e].t() + p["b1"][e]
            ys = ys.index_put((t, k), (torch.nn.functional.silu(z[:, :ffn]) * z[:, ffn:]) @ p["w2"][e].t() + p["b2"][e])
    (w.unsqueeze(2) * ys).sum(1).backward(dout.float())
    size = dout.float().norm(dim=1, keepdim=True) * ys.detach().norm(dim=2)
    w = w.detach()
    room = torch.zeros(tokens, experts, device="cuda").scatter_(1, idx, w * (size + (w * size).sum(1, keepdim=True)))
    return got, p["router"].grad, 6 * 0.08 * hidden ** -0.5 * room.t() @ xr.abs()


@pytest.mark.parametrize("shape", [(1, 256, 256, 4, 4), (2, 256, 512, 8, 3), (300, 512, 256, 8, 2)], ids=str)
def test_router_gradient_within_its_terms(moe_ffn, shape):
    for seed in range(60):
        got, want, bound = layer_and_autograd(moe_ffn, seed, *shape)
        assert ((got - want).abs() <= bound).all(), seed
