"""The projections' 64-bit oracle against automatic differentiation and plain loops."""
import pytest
import torch

from oracle import layers_ref as ref

ACTS = ("silu", "gelu", "gelu_tanh", "relu")


@pytest.mark.parametrize("name", ACTS)
def test_activations(name):
    g = torch.linspace(-6, 6, 401, dtype=torch.float64).requires_grad_()
    f = {"silu": torch.nn.functional.silu, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[name](g)
    a, d = ref.act(g.detach(), name)
    assert torch.allclose(a, f.detach(), atol=1e-13, rtol=1e-12)
    want, = torch.autograd.grad(f.sum(), g)
    inside = g.detach() != 0  # relu's kink: 0 here
    assert torch.allclose(d[inside], want[inside], atol=1e-13, rtol=1e-10)
    assert ref.act(torch.zeros(1, dtype=torch.float64), "relu")[1] == 0
    assert float(d.abs().max()) < 1.131  # what the bounds count with


def test_linear_row_by_row():
    torch.manual_seed(0)
    x, w = torch.randn(9, 12).bfloat16(), torch.randn(7, 12).bfloat16()
    a, b, s = torch.randn(3, 8, 12).bfloat16(), torch.randn(3, 7, 8).bfloat16(), torch.rand(3)
    index = torch.tensor([0, 1, -1, 2, 2, 5, 0, -9, 1])
    y, bound = ref.linear(x, w, a, b, s, index)
    for i in range(9):
        want = x[i].double() @ w.double().t()
        j = int(index[i])
        if 0 <= j < 3:
            want = want + float(s[j]) * (b[j].double() @ (a[j].double() @ x[i].double()))
        assert torch.allclose(y[i], want, rtol=1e-13, atol=1e-13)
        # Half a bf16 step of y, and less than 2^-13 of the terms' magnitudes: t's two parts
        # 2^-14, the sums (12 / 16 + 8) 2^-21 and 3 (28 / 16 + 8) 2^-21.
        size = x[i].abs().double() @ w.abs().double().t()
        if 0 <= j < 3:
            size = size + float(s[j]) * (b[j].abs().double() @ (a[j].abs().double() @ x[i].abs().double()))
        half = 2.0 ** -8 * y[i].abs()
        assert (bound[i] > half).all() and (bound[i] < half + 2.0 ** -13 * size).all()


@pytest.mark.parametrize("name", ACTS)
def test_gradients(name):
    torch.manual_seed(1)
    m, f, k = 5, 8, 6
    x, wi, wo = (torch.randn(*s).half() for s in ((m, k), (2 * f, k), (k, f)))
    dy = torch.randn(m, k).half()
    leaves = [t.double().requires_grad_() for t in (x, wi, wo)]
    pre = leaves[0] @ leaves[1].t()
    h = ref.act(pre[:, :f], name)[0] * pre[:, f:]
    want = torch.autograd.grad((h @ leaves[2].t() * dy.double()).sum(), leaves)
    got = ref.backward(x, wi, pre.detach(), name, dy=dy, w_out=wo)
    for t, n in zip(want, ("dx", "dw_in", "dw_out")):
        assert torch.allclose(got[n][0], t, rtol=1e-12, atol=1e-12)
        assert (got[n][1] > 0).all()
    hh, hb, p, pb = ref.gated(x, wi, name)
    assert torch.allclose(hh, h.detach(), rtol=1e-13) and torch.allclose(p, pre.detach(), rtol=1e-13)
    assert (hb >= 2.0 ** -11 * hh.abs()).all() and (pb >= 2.0 ** -11 * p.abs()).all()
    dh = (dy.double() @ wo.double()).half()
    got = ref.backward(x, wi, pre.detach(), name, dh=dh)
    want = torch.autograd.grad(
        ref.act((q := leaves[0] @ leaves[1].t())[:, :f], name)[0] * q[:, f:], leaves[:2], dh.double())
    for t, n in zip(want, ("dx", "dw_in")):
        assert torch.allclose(got[n][0], t, rtol=1e-12, atol=1e-12)
