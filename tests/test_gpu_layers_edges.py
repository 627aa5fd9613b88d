"""A layer's projections at the ends of their ranges, against the definitions in 64 bits
(oracle/layers_ref.py, which derives the bounds)."""
import pytest
import torch

from oracle import layers_ref as ref
from stream_decomposition_abft_gb300 import layers

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    w = layers.workspace()
    yield w
    torch.cuda.synchronize()
    assert w.report().timeouts == 0


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)


def check(got, want, bound, what=""):
    got = got.double()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    assert float(over.max()) <= 0, f"{what}: off by {float(over.max())} more than the bound"


# ------------------------------------------------------------------ a plan with no room left
# Each row its own adapter: 128 to a tile of single CTAs, 256 to one of the pairs, whose plan
# then ends with the last rows. With 1100 rows x 2560 columns the pairs run (50 tiles of 76
# pairs), with 256 and 300 rows single CTAs.
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 136, 512])
@pytest.mark.parametrize("s", [253, 254, 255, 256, 300, 1100])
def test_adapter_of_its_own_for_each_row_of_a_pair(ws, r, s):
    own_rows(ws, 1100, 2560, 136, r, s)


@pytest.mark.parametrize("r", [16, 24, 64, 136])
@pytest.mark.parametrize("m,s", [(127, 127), (128, 128), (256, 256), (255, 300), (300, 254)])
def test_adapter_of_its_own_for_each_row_of_a_cta(ws, m, s, r):
    own_rows(ws, m, 264, 200, r, s)


@pytest.mark.parametrize("m,n,k,s,r", [(256, 16384, 520, 256, 32), (512, 8192, 1032, 512, 24),
                                       (1024, 4096, 264, 1024, 64), (770, 4096, 1032, 254, 48)])
def test_adapter_of_its_own_for_each_row_at_serving_sizes(ws, m, n, k, s, r):
    own_rows(ws, m, n, k, r, s)


def own_rows(ws, m, n, k, r, s):
    g = gen(m + r + s)
    x, w = normal(g, m, k), normal(g, n, k, scale=k ** -0.5)
    a, b = normal(g, s, r, k, scale=k ** -0.5), normal(g, s, n, r, scale=r ** -0.5)
    f = 0.5 + torch.rand(s, generator=g, device="cuda")
    i = torch.arange(m, device="cuda") % s
    # The definition for the rows together: row i's adapter is s = i mod the stack.
    xd, wd = x.double(), w.double()
    y, size = xd @ wd.t(), xd.abs() @ wd.abs().t()
    u, least, acc = ref.U[x.dtype], ref.LEAST[x.dtype], ref.acc
    bound = acc(k) * size
    for at in range(0, m, 128):
        rows = torch.arange(at, min(at + 128, m), device="cuda")
        ai, bi, fi = a[i[rows]].double(), b[i[rows]].double(), f[i[rows]].double()[:, None]
        t = fi * torch.einsum("mk,mrk->mr", xd[rows], ai)
        off = fi * acc(k) * torch.einsum("mk,mrk->mr", xd[rows].abs(), ai.abs()) + \
            4 * u * u * t.abs() + least
        y[rows] += torch.einsum("mr,mnr->mn", t, bi)
        bound[rows] += torch.einsum("mr,mnr->mn", off, bi.abs()) + acc(k + 2 * r) * (
            size[rows] + 2 * torch.einsum("mr,mnr->mn", t.abs(), bi.abs()))
    got = layers.linear(x, w, layers.Adapters(a, b, f), i.int(), workspace=ws)
    check(got, y, bound + u * (y.abs() + bound) + least)


# ------------------------------------------------------------------ out beside its inputs
def test_out_in_a_buffer_of_its_inputs(ws):
    """Columns of one buffer: taken where they lie beside one another, refused where they share
    a byte."""
    from stream_decomposition_abft_gb300.skgemm import SkgError
    g = gen(12)
    m, n, k, r = 300, 72, 64, 16
    buf = normal(g, m, k + n + 8)
    w, i = normal(g, n, k), torch.zeros(m, dtype=torch.int32, device="cuda")
    ad = layers.Adapters(normal(g, 1, r, k), normal(g, 1, n, r))
    x = buf[:, :k]
    want, plain = layers.linear(x, w, ad, i, workspace=ws), layers.linear(x, w, workspace=ws)
    before = buf.clone()
    assert torch.equal(layers.linear(x, w, ad, i, out=buf[:, k:k + n], workspace=ws), want)
    assert torch.equal(layers.linear(x, w, out=buf[:, k + 8:], workspace=ws), plain)
    assert torch.equal(x, before[:, :k]) and torch.equal(buf[:, k:k + 8], want[:, :8])
    for out in (buf[:, k - 8:k - 8 + n], buf[:, :n]):
        with pytest.raises(SkgError, match="argument"):
            layers.linear(x, w, out=out, workspace=ws)
    with pytest.raises(SkgError, match="argument"):
        layers.linear(x[:8], w, out=torch.as_strided(w, (8, n), (n, 1)), workspace=ws)
    assert torch.equal(x, before[:, :k])


def test_autograd_sees_a_given_out_written(ws):
    from stream_decomposition_abft_gb300 import mx
    g = gen(13)
    x, w = normal(g, 8, 64), normal(g, 16, 64)
    a, b = mx.quantize(x, "mxfp8"), mx.quantize(w, "mxfp8")
    for write in (lambda out: layers.linear(x, w, out=out, workspace=ws),
                  lambda out: mx.matmul(a, b, out=out)):
        out = normal(g, 8, 16)
        p = torch.ones(8, 16, dtype=torch.bfloat16, device="cuda", requires_grad=True)
        loss = (p * out).sum()  # keeps out for p's gradient
        assert write(out) is out
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        with torch.inference_mode():
            kept = normal(g, 8, 16)
        assert write(kept) is kept  # an inference tensor has no version


# ------------------------------------------------------------------ the range of fp16
@pytest.mark.parametrize("size", [1e-4, 1e-6, 3e-8])
@pytest.mark.parametrize("m", [40, 129, 600])
def test_small_gradients_in_fp16(ws, m, size):
    """Between the products gradients are off by half a subnormal step (in the bound) at most."""
    g = gen(m)
    f, k = 136, 72
    x, w = normal(g, m, k, dtype=torch.float16), normal(g, 2 * f, k, dtype=torch.float16)
    wo, pre = normal(g, k, f, dtype=torch.float16), normal(g, m, 2 * f, dtype=torch.float16)
    dh, dy = normal(g, m, f, scale=size, dtype=torch.float16), \
        normal(g, m, k, scale=size, dtype=torch.float16)
    assert dh.any()
    want = ref.backward(x, w, pre, "silu", dh=dh)
    for what, t in zip(("dx", "dw_in"), layers.gated_backward(dh, x, w, pre, workspace=ws)):
        check(t, *want[what], what=what)
    want = ref.backward(x, w, pre, "silu", dy=dy, w_out=wo)
    for what, t in zip(("dx", "dw_in", "dw_out"),
                       layers.feed_forward_backward(dy, x, w, wo, pre, workspace=ws)):
        check(t, *want[what], what=what)


@pytest.mark.parametrize("m", [40, 300])
def test_large_gradients_in_fp16(ws, m):
    """A projection's gradient beyond 65504 is infinite: its token's dx is not finite, and other
    tokens' are right."""
    g = gen(m)
    f, k = 136, 72
    x, w = (normal(g, r, k, scale=1e-4, dtype=torch.float16) for r in (m, 2 * f))
    pre = normal(g, m, 2 * f, scale=4.0, dtype=torch.float16)
    dh = normal(g, m, f, scale=1500.0, dtype=torch.float16)
    dh[::2] *= 8
    a, da = ref.act(pre[:, :f].double(), "silu")
    dpre = torch.cat((dh.double() * pre[:, f:].double() * da, dh.double() * a), 1).abs()
    most = dpre.max(1).values
    fits, over = most < 65000, most > 66000
    assert fits.any() and over.any()
    dx, dw = layers.gated_backward(dh, x, w, pre, workspace=ws)
    want = ref.backward(x, w, pre, "silu", dh=dh)
    check(dx[fits], want["dx"][0][fits], want["dx"][1][fits])
    assert not torch.isfinite(dx[over]).all(1).any()
    fits, over = dpre.max(0).values < 65000, dpre.max(0).values > 66000
    check(dw[fits], want["dw_in"][0][fits], want["dw_in"][1][fits]) if fits.any() else None
    assert not torch.isfinite(dw[over]).all(1).any()


# ------------------------------------------------------------------ infinite weights
@pytest.mark.parametrize("m", [5, 40, 300])
def test_infinite_weights_are_never_finite(ws, m):
    """Infinities of a weight reach the results that they are a term of (as infinities or NaN:
    the operands in two parts may cancel), and no others."""
    g = gen(m)
    f, k, n, r = 72, 64, 136, 16
    x, w = normal(g, m, k), normal(g, n, k)
    a, b = normal(g, 2, r, k), normal(g, 2, n, r)
    i = (torch.arange(m, device="cuda") % 2).int()
    clean = layers.linear(x, w, layers.Adapters(a, b), i, workspace=ws)
    b[1, 7, 3] = float("inf")
    y = layers.linear(x, w, layers.Adapters(a, b), i, workspace=ws)
    assert not torch.isfinite(y[1::2, 7]).any()
    y[1::2, 7] = clean[1::2, 7]
    assert torch.equal(y, clean)

    wi, wo = normal(g, 2 * f, k), normal(g, k, f)
    pre, dy = normal(g, m, 2 * f), normal(g, m, k)
    clean = layers.feed_forward_backward(dy, x, wi, wo, pre, "gelu", workspace=ws)
    wi[70, 5] = float("-inf")
    dx, dwi, dwo = layers.feed_forward_backward(dy, x, wi, wo, pre, "gelu", workspace=ws)
    assert not torch.isfinite(dx[:, 5]).any()
    dx[:, 5] = clean[0][:, 5]
    for got, want in zip((dx, dwi, dwo), clean):
        assert torch.equal(got, want)


# ------------------------------------------------------------------ far gates, few rows
@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("m", [11, 16, 100, 128])
def test_far_gates_of_few_rows(ws, name, m):
    """All of the far gates in the path of few rows and in gradients held in two parts."""
    far = torch.tensor([0.0, 1e-30, -1e-30, 30.0, -30.0, 100.0, -100.0, 1e4, -1e4, 1e18, -1e18],
                       device="cuda").bfloat16()
    k, f = 8, 16
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = far[torch.arange(m, device="cuda") % len(far)]
    w = torch.zeros(2 * f, k, dtype=torch.bfloat16, device="cuda")
    w[:f, 0], w[f:, 1], x[:, 1] = 1.0, 1.0, 0.5
    h, pre = layers.gated(x, w, name, save=True, workspace=ws)
    want, bound, wp, pb = ref.gated(x, w, name)
    check(h, want, bound + 1e-30)
    check(pre, wp, pb)
    dh = torch.ones(m, f, dtype=torch.bfloat16, device="cuda")
    grads = ref.backward(x, w, pre, name, dh=dh)
    dx, dw = layers.gated_backward(dh, x, w, pre, name, workspace=ws)
    check(dx, *grads["dx"])
    check(dw, *grads["dw_in"])
