"""One Mixture-of-Experts feed-forward layer, trained for a few steps with this library.

The layer is ``out = hidden + sum_k w[t, k] * expert_{e(t, k)}(hidden)`` with SwiGLU experts:
a router picks top_k experts per token, the tokens' rows are sorted by expert, the experts'
two products run in MXFP8 (bias, activation and the saved pre-activation in the product's
epilogue), and the rows come back to token order weighted.  The backward pass covers every
parameter: expert weights and biases, router, and the layer's input.

    python examples/moe_ffn.py [--steps N] [--tokens T]

Only the router's small projection (hidden x experts) uses a torch product; everything else is
a call of moe_grouped_gemm_wgrad_gb300.mgw.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from moe_grouped_gemm_wgrad_gb300 import mgw  # noqa: E402


class MoeFfn:
    """Parameters in fp32, products on MXFP8 copies that :meth:`quantize_weights` makes once per
    step.  ``hidden`` must be a multiple of 256, ``ffn`` (columns after the gate) too."""

    def __init__(self, hidden: int, ffn: int, experts: int, top_k: int, seed: int = 0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def init(*shape, fan_in):
            return torch.randn(*shape, generator=g, device=device) * fan_in ** -0.5

        self.hidden, self.ffn, self.experts, self.top_k = hidden, ffn, experts, top_k
        self.router = init(experts, hidden, fan_in=hidden)
        self.w1 = init(experts, 2 * ffn, hidden, fan_in=hidden)   # gate rows, then up rows
        self.w2 = init(experts, hidden, ffn, fan_in=ffn)
        self.b1 = torch.zeros(experts, 2 * ffn, device=device)
        self.b2 = torch.zeros(experts, hidden, device=device)
        self.off1 = torch.arange(experts + 1, device=device, dtype=torch.int32) * (2 * ffn)
        self.off2 = torch.arange(experts + 1, device=device, dtype=torch.int32) * hidden
        self.status = torch.zeros(1, device=device, dtype=torch.int32)
        self.quantize_weights()

    def parameters(self):
        return {"router": self.router, "w1": self.w1, "w2": self.w2, "b1": self.b1, "b2": self.b2}

    def quantize_weights(self) -> None:
        """MXFP8 copies along both axes: rows for the forward products, transposed for the data
        gradients."""
        w1 = self.w1.bfloat16().view(-1, self.hidden)
        w2 = self.w2.bfloat16().view(-1, self.ffn)
        self.w1_fwd = mgw.mxfp8_quantize_rows(w1, self.off1)
        self.w2_fwd = mgw.mxfp8_quantize_rows(w2, self.off2)
        self.w1_bwd = mgw.mxfp8_quantize(w1, self.off1)
        self.w2_bwd = mgw.mxfp8_quantize(w2, self.off2)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """out [T, hidden] bf16 from x [T, hidden] bf16; keeps what the backward pass needs."""
        st = self.status
        logits = x.float() @ self.router.t()
        idx, weights = mgw.moe_route(logits, self.top_k, status=st)
        off, row_index, row_of = mgw.moe_dispatch(idx, self.experts, status=st)
        rows = x.shape[0] * self.top_k   # nothing is masked here, so no pair is dropped
        xq, xs = mgw.mxfp8_quantize_rows(x, off, row_index=row_index, status=st)
        h, z = mgw.grouped_fprop_mxfp8_act(xq, xs, *self.w1_fwd, off, rows, 2 * self.ffn,
                                           mgw.ACT_SWIGLU, bias=self.b1, save_preact=True, status=st)
        hq, hs = mgw.mxfp8_quantize_rows(h, off, status=st)
        y = mgw.grouped_fprop_mxfp8_act(hq, hs, *self.w2_fwd, off, rows, self.hidden, mgw.ACT_NONE,
                                        bias=self.b2, status=st)
        out = mgw.moe_combine(y, row_of, weights=weights, residual=x, status=st)
        self.saved = (x, logits, idx, weights, off, row_index, row_of, z, h, y)
        return out

    def backward(self, dout: torch.Tensor):
        """(dx [T, hidden] bf16, gradients by parameter name) from dout [T, hidden] bf16."""
        x, logits, idx, weights, off, row_index, row_of, z, h, y = self.saved
        st, rows = self.status, y.shape[0]
        grads = {}
        dy, dweights = mgw.moe_combine_backward(dout, y, row_of, weights=weights, status=st)
        # second product: bias, weights, data
        _, grads["b2"] = mgw.grouped_act_backward(dy, None, off, mgw.ACT_NONE, with_dbias=True, status=st)
        gq, gs = mgw.mxfp8_quantize(dy, off, status=st)
        hq, hs = mgw.mxfp8_quantize(h, off, status=st)
        grads["w2"] = mgw.grouped_wgrad_mxfp8(gq, gs, hq, hs, off, rows, status=st).view_as(self.w2)
        dyq, dys = mgw.mxfp8_quantize_rows(dy, off, status=st)
        dh = mgw.grouped_dgrad_mxfp8(dyq, dys, *self.w2_bwd, off, rows, status=st)
        # activation and first bias, then the first product
        dz, grads["b1"] = mgw.grouped_act_backward(dh, z, off, mgw.ACT_SWIGLU, with_dbias=True, status=st)
        gq, gs = mgw.mxfp8_quantize(dz, off, status=st)
        xq, xs = mgw.mxfp8_quantize_gather(x, row_index, off, status=st)
        grads["w1"] = mgw.grouped_wgrad_mxfp8(gq, gs, xq, xs, off, rows, status=st).view_as(self.w1)
        dzq, dzs = mgw.mxfp8_quantize_rows(dz, off, status=st)
        dx_rows = mgw.grouped_dgrad_mxfp8(dzq, dzs, *self.w1_bwd, off, rows, status=st)
        # back to tokens: the gather's gradient, the residual's, the router's
        dx = mgw.moe_combine(dx_rows, row_of, residual=dout, status=st)
        dlogits = mgw.moe_route_backward(logits, idx, dweights, status=st)
        grads["router"] = dlogits.t() @ x.float()
        dx = (dx.float() + dlogits @ self.router).bfloat16()
        return dx, grads

    def step(self, grads, lr: float) -> None:
        for name, p in self.parameters().items():
            p.sub_(grads[name].float(), alpha=lr)
        self.quantize_weights()


def train(steps: int = 20, tokens: int = 2048, hidden: int = 512, ffn: int = 256, experts: int = 16,
          top_k: int = 4, lr: float = 0.2, seed: int = 0):
    """Fits the layer to a fixed random map by gradient descent; returns the losses."""
    layer = MoeFfn(hidden, ffn, experts, top_k, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    target = x.float() + torch.tanh(x.float() @ torch.randn(hidden, hidden, generator=g, device="cuda")
                                    * hidden ** -0.5)
    losses = []
    for _ in range(steps):
        out = layer.forward(x)
        diff = out.float() - target
        losses.append(0.5 * diff.square().sum(1).mean())
        # gradient of the mean over tokens, scaled up so that bf16 holds it well
        _, grads = layer.backward(diff.bfloat16())
        layer.step({k: v / tokens for k, v in grads.items()}, lr)
    if int(layer.status.item()) != 0:
        raise RuntimeError(f"device status {int(layer.status.item())}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--tokens", type=int, default=2048)
    a = p.parse_args()
    for i, loss in enumerate(train(a.steps, a.tokens)):
        print(f"step {i:3d}  loss {loss:.4f}")
