"""The projections' activations and their derivatives in fp32, element by element against
their definitions in 64 bits.

Bounds, from the errors that CUDA states for what the kernels call: e^x by __expf is off by
(2 + 1.173 |x|) 2^-23 of its value, a quotient by __fdividef by 2 2^-23, another operation by
2^-24. Below 2^-126 numbers are 2^-149 apart, so a result or an intermediate there is off by
half of that whatever its value: LEAST is added once for each.
"""
import math

import pytest
import torch

from oracle import layers_ref as ref
from stream_decomposition_abft_gb300 import layers, skgemm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24  # half a step
LEAST = 2.0 ** -150  # half a step of the subnormal numbers


def values():
    far = torch.linspace(-130, 130, 520001, dtype=torch.float64)
    near = torch.linspace(-14, 14, 560001, dtype=torch.float64)
    small = 2.0 ** torch.linspace(-140, 2, 20001, dtype=torch.float64)
    large = 2.0 ** torch.linspace(2, 127, 4001, dtype=torch.float64)
    return torch.cat((far, near, small, -small, large, -large, torch.zeros(1))).float().cuda()


def run(name, g):
    a, d = torch.full_like(g, 7.0), torch.full_like(g, 7.0)
    st = skgemm.layers_test_activation(layers.ACTIVATIONS[name], g.numel(), g.data_ptr(),
                                       a.data_ptr(), d.data_ptr(),
                                       torch.cuda.current_stream().cuda_stream)
    assert st == skgemm.OK
    return a, d


def exp_err(x):
    return (2 + 1.173 * x.abs()) * 2 * U


def sigmoid(x):
    """(p, its error), of an x that is exact."""
    e = torch.exp(-x.abs())
    p = torch.where(x >= 0, 1 / (1 + e), e / (1 + e))
    # The exponential's error counts in full below 0 (where 1 + e loses some of it), by
    # e / (1 + e) above.
    rel = exp_err(x) * torch.where(x >= 0, e / (1 + e), torch.ones_like(e))
    return p, p * (rel + 4 * U + 2 * U) + 4 * LEAST


def bounds(name, g):
    """(a, its error, d, its error) for g in 64 bits."""
    s = g.abs()
    if name == "silu":
        p, off = sigmoid(g)
        q = 1 / (1 + torch.exp(g))  # 1 - p
        a, d = g * p, p + g * p * q
        d_off = off * (1 + s * q) + p * s * (off + U) + 4 * U * (p + s * p * q)
        return a, s * off + U * a.abs() + LEAST, d, d_off + 4 * LEAST
    if name == "gelu":
        z = s / math.sqrt(2)
        r = torch.special.erfc(z)  # of |x|
        # x is off by 2 U of itself (erfc' / erfc is below 2 z + 1.2), z^2 by another U. The
        # polynomial of t: its fit by 0.7 U, its sum (terms of at most half of it) by 6 U, t's
        # 4 U by up to 2.26 times as much (d ln(e^z^2 erfc z) / d ln t at z = 0), two products.
        rel = (2 * z + 1.2) * z * 2 * U + z * z * U + exp_err(z * z) + 18 * U
        p = torch.where(g >= 0, 1 - r / 2, r / 2)
        off = r / 2 * rel + 2 * U * p + 4 * LEAST
        pdf = torch.exp(-s * s / 2) / math.sqrt(2 * math.pi)
        pdf_off = pdf * (s * s / 2 * U + exp_err(s * s / 2) + 4 * U) + 4 * LEAST
        return g * p, s * off + U * s * p + LEAST, p + g * pdf, \
            off + s * pdf_off + 2 * U * (p + s * pdf) + 4 * LEAST
    if name == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        t = s.clamp_max(1e3)  # (d is 0 or 1 long before)
        w = (k * (g + 0.044715 * g ** 3)).clamp(-1e9, 1e9)
        p, off = sigmoid(w)
        q = 1 / (1 + torch.exp(w))
        off = off + p * q * w.abs() * 6 * U  # w's own error
        c = k * (1 + 3 * 0.044715 * t * t)
        d = torch.where(p * q == 0, p, p + g.clamp(-1e3, 1e3) * p * q * c)
        # q = p (1 - p) of the computed p: off by |1 - 2 p| of p's error and by p 2 U; where it
        # is 0 the term is left out, which is off by no more.
        d_off = off + t * c * (off + 2 * U * p) * (w < 20) + 8 * U * (p + t * p * q * c)
        return g * p, s * off + U * s * p + LEAST, d, d_off + 4 * LEAST
    a, d = ref.act(g, name)
    return a, 0 * a, d, 0 * d


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu"])
def test_against_the_definition(name):
    g = values()
    a, d = run(name, g)
    want, off, want_d, off_d = bounds(name, g.double())
    for what, got, w, o in (("act", a, want, off), ("act'", d, want_d, off_d)):
        assert torch.isfinite(got).all(), what
        over = (got.double() - w).abs() - o
        i = int(over.argmax())
        assert float(over[i]) <= 0, \
            f"{what}({float(g[i])}) = {float(got[i])}, not {float(w[i])} to {float(o[i])}"


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_far_gates_keep_their_bits(name):
    """Down to the least normal results no value is lost."""
    at = -88.0 if name == "silu" else -10.05
    g = torch.linspace(at, at / 2, 2001).cuda()
    a, _ = run(name, g)
    want = ref.act(g.double(), name)[0]
    assert float(want.abs().min()) > 2.0 ** -126
    assert float(((a.double() - want) / want).abs().max()) < 2.0 ** -14


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu"])
def test_infinities_and_nan(name):
    g = torch.tensor([float("inf"), float("nan")], device="cuda")
    a, d = run(name, g)
    assert float(a[0]) == float("inf") and a[1].isnan() and d[1].isnan()


def test_arguments():
    assert skgemm.layers_test_activation(4, 0, None, None, None, None) == skgemm.ERR_ARG
    assert skgemm.layers_test_activation(0, -1, None, None, None, None) == skgemm.ERR_ARG
    assert skgemm.layers_test_activation(0, 1, None, None, None, None) == skgemm.ERR_ARG
    assert skgemm.layers_test_activation(0, 0, None, None, None, None) == skgemm.OK
