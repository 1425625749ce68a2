"""The example layer (examples/moe_ffn.py), which runs every routed-layer operator together,
against autograd on the same parameters in fp32.

Tolerance: e4m3 keeps three mantissa bits, a relative rounding error of about 2.6% rms, so a
product of two quantized operands is off by 3.7% of its rms, and two chained products with
what they pass on by 5 to 8%; every tensor is held to 12% of its rms over all elements.  The
router's choice is compared exactly (both see the same fp32 logits)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def moe_ffn():
    spec = importlib.util.spec_from_file_location("moe_ffn", os.path.join(ROOT, "examples", "moe_ffn.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rms_error(got, want):
    return float((got.float() - want).square().mean().sqrt() / want.square().mean().sqrt())


@pytest.mark.parametrize("tokens,hidden,ffn,experts,top_k", [(300, 512, 256, 8, 2), (1, 256, 256, 4, 4),
                                                             (777, 256, 512, 32, 6)])
def test_layer_matches_autograd(moe_ffn, tokens, hidden, ffn, experts, top_k):
    layer = moe_ffn.MoeFfn(hidden, ffn, experts, top_k, seed=tokens)
    layer.b1.normal_(std=0.3)
    layer.b2.normal_(std=0.3)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    dout = torch.randn(tokens, hidden, device="cuda").bfloat16()
    out = layer.forward(x)
    dx, grads = layer.backward(dout)
    assert int(layer.status.item()) == 0

    p = {k: v.clone().requires_grad_() for k, v in layer.parameters().items()}
    xr = x.float().requires_grad_()
    logits = xr @ p["router"].t()
    idx = layer.saved[2].long()
    assert torch.equal(idx, torch.topk(layer.saved[1], top_k).indices)
    w = torch.softmax(logits.gather(1, idx), 1)
    want = xr
    for e in range(experts):
        t, k = (idx == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        z = xr[t] @ p["w1"][e].t() + p["b1"][e]
        h = torch.nn.functional.silu(z[:, :ffn]) * z[:, ffn:]
        y = h @ p["w2"][e].t() + p["b2"][e]
        want = want.index_add(0, t, w[t, k].unsqueeze(1) * y)
    want.backward(dout.float())
    assert _rms_error(out, want.detach()) < 0.12
    assert _rms_error(dx, xr.grad) < 0.12
    for name, v in p.items():
        assert _rms_error(grads[name], v.grad) < 0.12, name


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 4, 4), (3, 8, 2), (65, 16, 5)])
def test_router_gradient_of_the_layer_from_its_own_rows(moe_ffn, tokens, experts, top_k):
    """The router's gradient against 64 bits on the expert outputs that the layer itself kept: of few
    tokens it is a difference of nearly equal numbers, in which the quantization of those outputs
    weighs more than in the other gradients.  Held to fp32's rounding of the terms before they
    cancel: 256-term dot products (2^-24 * (256 / 8 + 16), as combine's), and a few roundings."""
    layer = moe_ffn.MoeFfn(256, 256, experts, top_k, seed=3)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x, dout = (torch.randn(tokens, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    layer.forward(x)
    _, grads = layer.backward(dout)
    _, logits, idx, _, _, _, row_of, _, _, y = layer.saved
    dw = (y.double()[row_of.long()] * dout.double().unsqueeze(1)).sum(2)
    mag = (y.double()[row_of.long()] * dout.double().unsqueeze(1)).abs().sum(2)
    p = torch.softmax(logits.double().gather(1, idx.long()), 1)

    def to_experts(d):
        return torch.zeros(tokens, experts, dtype=torch.float64, device="cuda").scatter_(1, idx.long(), d)

    want = to_experts(p * (dw - (p * dw).sum(1, keepdim=True))).t() @ x.double()
    room = to_experts(p * (mag + (p * mag).sum(1, keepdim=True))).t() @ x.double().abs()
    # the fp32 library product that sums over the tokens rounds at most once per term
    tol = (2.0 ** -24 * (256 / 8 + 16) + 2.0 ** -24 * (tokens + 64)) * room
    assert ((grads["router"].double() - want).abs() <= tol).all()


def test_training_reduces_the_loss(moe_ffn):
    losses = moe_ffn.train(steps=12, tokens=1024)
    assert all(b < a for a, b in zip(losses, losses[1:]))
    assert losses[-1] < 0.9 * losses[0]
