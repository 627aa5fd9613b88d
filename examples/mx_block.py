"""A feed-forward block with microscaled products, forward and backward.

    h = x + residual;  u = rmsnorm(h) W1^T;  y = relu(u)^2 W2^T

The norm writes the first product's quantised operand itself; the second product
quantises its input. The backward pass runs both linear layers' gradients on
quantised operands and the norm's gradient on the stored sum. Compares with the
same block in fp32 and prints the relative errors.

    python examples/mx_block.py [--tokens 512] [--width 1024] [--hidden 2816] [--format mxfp8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from stream_decomposition_abft_gb300 import mx  # noqa: E402

EPS = 1e-5


def scale_of(t, fmt):
    """nvfp4's fp32 scale of a tensor."""
    return (t.float().abs().amax() / (448 * 6)).reshape(1) if fmt == "nvfp4" else None


class Block:
    """Weights in bf16, quantised once for the forward and once for the backward."""

    def __init__(self, norm, w1, w2, fmt):
        self.norm, self.fmt, self.ws = norm, fmt, mx.workspace(norm.device)
        self.w1, self.w1t = mx.quantize_both(w1, fmt, tensor_scale=scale_of(w1, fmt))
        self.w2, self.w2t = mx.quantize_both(w2, fmt, tensor_scale=scale_of(w2, fmt))

    def forward(self, x, residual, norm_scale=None):
        q, h, rstd = mx.rmsnorm(x, self.norm, EPS, residual=residual, format=self.fmt,
                                tensor_scale=norm_scale)
        u = mx.matmul(q, self.w1, workspace=self.ws)
        a = torch.relu(u).square()
        y = mx.linear(a, self.w2, tensor_scale=scale_of(a, self.fmt), workspace=self.ws)
        return y, (h, rstd, u, a)

    def backward(self, dy, saved):
        """(dx = dresidual, dnorm, dW1, dW2); the sum h also leaves the block as it is
        (the residual path), with gradient dy here."""
        h, rstd, u, a = saved
        f = self.fmt
        at = mx.quantize(a, f, transpose=True, tensor_scale=scale_of(a, f))
        da, dw2 = mx.linear_backward(dy, self.w2t, at, tensor_scale=scale_of(dy, f),
                                     workspace=self.ws)
        du = da * 2 * torch.relu(u)
        n = (h.float() * rstd[:, None] * self.norm.float()).to(h.dtype)
        nt = mx.quantize(n, f, transpose=True, tensor_scale=scale_of(n, f))
        dn, dw1 = mx.linear_backward(du, self.w1t, nt, tensor_scale=scale_of(du, f),
                                     workspace=self.ws)
        dx, dnorm = mx.rmsnorm_backward(dn, h, self.norm, rstd, dresidual=dy)
        return dx, dnorm, dw1, dw2


def run(tokens, width, hidden, fmt, seed=0):
    """Relative errors {name: error} of the block's outputs against fp32."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s, scale=1.0: (scale * torch.randn(*s, generator=g, device="cuda")).bfloat16()
    x, residual, dy = rand(tokens, width), rand(tokens, width), rand(tokens, width)
    norm = rand(width, scale=0.1) + 1
    w1, w2 = rand(hidden, width, scale=width ** -0.5), rand(width, hidden, scale=hidden ** -0.5)
    block = Block(norm, w1, w2, fmt)
    # nvfp4's scale of the norm's output: calibrated, here from one look at it.
    h = x.float() + residual.float()
    n = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * norm.float()
    y, saved = block.forward(x, residual, scale_of(n, fmt))
    grads = block.backward(dy, saved)
    if block.ws.report().timeouts:
        raise RuntimeError("a device-side wait ran out")

    ref = [t.float().requires_grad_() for t in (x, norm, w1, w2)]
    h = ref[0] + residual.float()
    n = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * ref[1]
    want = torch.relu(n @ ref[2].t()).square() @ ref[3].t()
    want_grads = torch.autograd.grad((want * dy.float()).sum() + (h * dy.float()).sum(), ref)
    pairs = [("y", y, want)] + list(zip(("dx", "dnorm", "dW1", "dW2"), grads, want_grads))
    return {k: float((a.float() - b.detach()).norm() / b.detach().norm()) for k, a, b in pairs}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=2816)
    ap.add_argument("--format", default="mxfp8", choices=list(mx.FORMATS))
    a = ap.parse_args()
    for name, err in run(a.tokens, a.width, a.hidden, a.format).items():
        print(f"{name:6s} relative error against fp32: {err:.4f}")
