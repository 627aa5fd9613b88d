"""A layer's projections from their definitions, in 64 bits on the CPU or the inputs' device,
with bounds on what a computation in 32 bits with results of `kind` may differ by.

A bound counts: half a step of the result's type (u), half a step of each intermediate that is
rounded to fewer bits, and the sums. A tensor-core instruction adds 16 products to the
accumulator with an error of at most 2^-21 of the sum of their magnitudes (the terms are
aligned to the largest and cut), so a sum of k products is off by at most (k / 16 + 8) 2^-21
of its terms' magnitudes (the 8: partial sums joined at the end). The activations are off by
2^-18 of their value (exponentials of arguments up to 2^6 with 2^-24 of the argument).
"""
from __future__ import annotations

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half a subnormal step
ACT_ERR = 2.0 ** -18


def acc(k: int) -> float:
    return (k / 16 + 8) * 2.0 ** -21


def act(g, name):
    """(act(g), act'(g))."""
    if name == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        p = torch.sigmoid(2 * k * (g + 0.044715 * g ** 3))
        return g * p, p + g * p * (1 - p) * 2 * k * (1 + 3 * 0.044715 * g * g)
    return g.clamp_min(0), (g > 0).to(g.dtype)


def linear(x, w, down=None, up=None, scale=None, index=None):
    """(y, bound)"""
    kind, k = x.dtype, x.shape[1]
    u = U[kind]
    x, w = x.double(), w.double()
    y, size = x @ w.t(), x.abs() @ w.abs().t()
    bound = acc(k) * size
    if down is not None:
        for s in range(down.shape[0]):
            rows = torch.nonzero(index == s)[:, 0]
            if not len(rows):
                continue
            f = 1.0 if scale is None else float(scale[s])
            a, b = down[s].double(), up[s].double()
            t = f * (x[rows] @ a.t())
            # t: its sum, and rounded to two parts.
            off = abs(f) * acc(k) * (x[rows].abs() @ a.abs().t()) + 4 * u * u * t.abs() + LEAST[kind]
            y[rows] += t @ b.t()
            bound[rows] += off @ b.abs().t() + \
                acc(k + 2 * a.shape[0]) * (size[rows] + 2 * t.abs() @ b.abs().t())
    return y, bound + u * (y.abs() + bound) + LEAST[kind]


def gated(x, w_in, name):
    """(h, bound of h, pre, bound of pre)"""
    kind, k = x.dtype, x.shape[1]
    u = U[kind]
    x, w = x.double(), w_in.double()
    pre, off = x @ w.t(), acc(k) * (x.abs() @ w.abs().t())
    f = pre.shape[1] // 2
    g, p = pre[:, :f], pre[:, f:]
    a, _ = act(g, name)
    h = a * p
    # |act'| <= 1.13, |act''| <= 1.2: the second-order part is in the 2.
    bound = 2 * off[:, :f] * p.abs() + (a.abs() + 2 * off[:, :f]) * off[:, f:] + ACT_ERR * (
        h.abs() + (g.abs() * p.abs() * 2.0 ** -6))
    return h, bound + u * (h.abs() + bound) + LEAST[kind], pre, off + u * (pre.abs() + off) + LEAST[kind]


def _dpre(dh, dh_off, pre, name, u, least):
    """(dpre, its bound, h, its bound) of gradients dh known to dh_off."""
    f = dh.shape[1]
    g, p = pre[:, :f], pre[:, f:]
    a, da = act(g, name)
    d = torch.cat((dh * p * da, dh * a), 1)
    slack = ACT_ERR * torch.cat((dh.abs() * p.abs() * (da.abs() + 1), dh.abs() * (a.abs() + g.abs() * 2.0 ** -6)), 1)
    off = torch.cat((dh_off * p.abs() * 1.13, dh_off * (a.abs() + 2.0 ** -10)), 1) + slack
    h = a * p
    h_off = ACT_ERR * (h.abs() + g.abs() * p.abs() * 2.0 ** -6)
    return d, off + u * (d.abs() + off) + least, h, h_off + u * (h.abs() + h_off) + least


def _product(a, a_off, b, b_off, kind):
    """(a b, bound) of factors known to a_off, b_off."""
    k = a.shape[1]
    y = a @ b
    bound = a_off @ b.abs() + a.abs() @ b_off + a_off @ b_off + 2 * acc(2 * k) * (a.abs() @ b.abs())
    return y, bound + U[kind] * (y.abs() + bound) + LEAST[kind]


def backward(x, w_in, pre, name, dh=None, dy=None, w_out=None):
    """{name: (gradient, bound)}: from dh, or from dy through w_out."""
    kind = x.dtype
    u = U[kind] if x.shape[0] > 128 else 4 * U[kind] ** 2  # kept in two parts up to 128 rows
    x, w = x.double(), w_in.double()
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    if dh is None:
        dy, wo = dy.double(), w_out.double()
        dh, off = dy @ wo, acc(dy.shape[1]) * (dy.abs() @ wo.abs())
    else:
        dh, off = dh.double(), zero * dh.double()
    d, d_off, h, h_off = _dpre(dh, off, pre.double(), name, u, LEAST[kind])
    out = dict(dx=_product(d, d_off, w, zero * w, kind),
               dw_in=_product(d.t(), d_off.t(), x, zero * x, kind))
    if w_out is not None:
        out["dw_out"] = _product(dy.t(), zero * dy.t(), h, h_off, kind)
    return out
