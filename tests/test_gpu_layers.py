"""A layer's projections on the GPU against their definitions in 64 bits (oracle/layers_ref.py,
which derives the bounds)."""
import pytest
import torch

from oracle import layers_ref as ref
from stream_decomposition_abft_gb300 import layers, mx

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


@pytest.fixture(scope="module")
def ws():
    w = layers.workspace()
    yield w
    torch.cuda.synchronize()
    assert w.report().timeouts == 0


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, kind, *shape, scale=1.0, pad=0):
    """Normal values; `pad` more elements from row to row, NaN."""
    t = torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(TYPES[kind])
    if not pad:
        return t
    buf = torch.full((*shape[:-1], shape[-1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    buf[..., :shape[-1]] = t
    return buf[..., :shape[-1]]


def rows16(g, kind, rows, cols, scale=1.0):
    """Rows on 16-byte boundaries."""
    return normal(g, kind, rows, cols, scale=scale, pad=-cols % 8)


def check(got, want, bound, what=""):
    got = got.double()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{what}: off by {worst} more than the bound {float(bound.max())}"


# ------------------------------------------------------------------ the plain projection
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 1), (1, 8, 64), (1, 1000, 8192), (3, 130, 72), (16, 256, 520), (17, 127, 65),
    (64, 1000, 2200), (128, 128, 64), (129, 257, 1000), (255, 640, 136), (256, 256, 256),
    (333, 1000, 2200), (513, 2049, 200), (1024, 1024, 1024), (2000, 3000, 320), (700, 5000, 1000)])
def test_linear(ws, kind, m, n, k):
    g = gen(m + n + k)
    x, w = rows16(g, kind, m, k), rows16(g, kind, n, k, k ** -0.5)
    check(layers.linear(x, w, workspace=ws), *ref.linear(x, w))


def test_linear_strides_and_out(ws):
    g = gen(1)
    x, w = normal(g, "bf16", 300, 200, pad=24), normal(g, "bf16", 520, 200, pad=56)
    buf = torch.full((302, 600), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:301, 8:528]
    got = layers.linear(x, w, out=out, workspace=ws)
    assert got.data_ptr() == out.data_ptr()
    check(out, *ref.linear(x, w))
    edge = buf.clone()
    edge[1:301, 8:528] = 7.0
    assert (edge == 7.0).all()
    # Columns whose number is no multiple of 8, on either kernel.
    for m in (5, 300, 2000):
        x = normal(g, "bf16", m, 64)
        w = normal(g, "bf16", 1003, 64)
        buf = torch.full((m, 1016), 7.0, dtype=torch.bfloat16, device="cuda")
        layers.linear(x, w, out=buf[:, :1003], workspace=ws)
        check(buf[:, :1003], *ref.linear(x, w))
        assert (buf[:, 1003:] == 7.0).all()


# ------------------------------------------------------------------ adapters
def stack(g, kind, s, r, n, k):
    return normal(g, kind, s, r, k, scale=k ** -0.5), normal(g, kind, s, n, r, scale=r ** -0.5), \
        0.5 + torch.rand(s, generator=g, device="cuda")


def indices(g, m, s, order):
    i = torch.randint(-1, s, (m,), generator=g, device="cuda")
    if order == "own":
        i = torch.arange(m, device="cuda") % s
    elif order == "segments":
        i = i.sort().values
    elif order == "none":
        i = torch.full_like(i, -1)
    elif order == "one":
        i = torch.full_like(i, s - 1)
    elif order == "last":  # the tile's last row alone
        i = torch.where(torch.arange(m, device="cuda") == m - 1, 0, -1)
    return i.int()


@pytest.mark.parametrize("order", ["mixed", "own", "segments", "none", "one", "last"])
@pytest.mark.parametrize("m", [1, 16, 40, 129, 300])
def test_adapters_orders(ws, m, order):
    g = gen(m)
    k, n, s, r = 520, 392, 150, 16
    x, w = normal(g, "bf16", m, k), normal(g, "bf16", n, k, scale=k ** -0.5)
    a, b, f = stack(g, "bf16", s, r, n, k)
    i = indices(g, m, s, order)
    y = layers.linear(x, w, layers.Adapters(a, b, f), i, workspace=ws)
    check(y, *ref.linear(x, w, a, b, f, i), what=order)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 48, 64, 72, 96, 128, 136, 200, 264, 512])
@pytest.mark.parametrize("m,n,k", [(9, 264, 328), (257, 136, 1000), (1100, 2560, 136)])
def test_adapters_ranks(ws, kind, r, m, n, k):
    g = gen(r + m)
    s = 11
    x, w = normal(g, kind, m, k), normal(g, kind, n, k, scale=k ** -0.5)
    a, b, f = stack(g, kind, s, r, n, k)
    i = indices(g, m, s, "mixed")
    y = layers.linear(x, w, layers.Adapters(a, b, f), i, workspace=ws)
    check(y, *ref.linear(x, w, a, b, f, i))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,s,r", [(1, 16, 16), (1, 3, 128), (2, 64, 64), (8, 64, 8), (7, 8, 16),
                                   (16, 2, 64), (16, 1, 128), (5, 4, 32), (13, 3, 40), (64, 5, 16),
                                   (128, 1, 128), (129, 8, 16), (300, 2, 64), (300, 8, 8),
                                   (200, 3, 40), (40, 4, 24), (333, 1, 96), (127, 2, 48),
                                   (16, 16, 8), (140, 16, 8), (9, 16, 8), (200, 5, 24), (65, 13, 8),
                                   (1, 5, 120)])
@pytest.mark.parametrize("n,k", [(1000, 2200), (264, 72), (128, 8), (3000, 1032)])
def test_adapters_few(ws, kind, m, s, r, n, k):
    """Few adapters to a tile (one launch), k split and not, rows with none."""
    g = gen(m + s)
    x, w = normal(g, kind, m, k), normal(g, kind, n, k, scale=k ** -0.5)
    a, b, f = stack(g, kind, s, r, n, k)
    for order in ("mixed", "none", "last"):
        i = indices(g, m, s, order)
        y = layers.linear(x, w, layers.Adapters(a, b, f), i, workspace=ws)
        check(y, *ref.linear(x, w, a, b, f, i), what=order)


@pytest.mark.parametrize("m,order", [(64, "mixed"), (333, "mixed"), (2048, "segments"), (2048, "own"),
                                     (2500, "mixed")])
def test_adapters_sizes(ws, m, order):
    g = gen(m)
    k, n, s, r = 2200, 1000, 64, 16
    if m > 2000:
        k, n = 512, 4096  # pairs
    x, w = normal(g, "bf16", m, k), normal(g, "bf16", n, k, scale=k ** -0.5)
    a, b, f = stack(g, "bf16", s, r, n, k)
    i = indices(g, m, s, order)
    y = layers.linear(x, w, layers.Adapters(a, b, f), i, workspace=ws)
    check(y, *ref.linear(x, w, a, b, f, i))


def test_adapters_strides_and_no_scale(ws):
    g = gen(3)
    m, k, n, s, r = 70, 200, 120, 6, 24
    x, w = normal(g, "f16", m, k, pad=8), normal(g, "f16", n, k)
    a = normal(g, "f16", 2 * s, r + 3, k, pad=16)[::2, :r]
    b = normal(g, "f16", s, n + 1, r, pad=40)[:, :n]
    i = indices(g, m, s, "mixed")
    y = layers.linear(x, w, layers.Adapters(a, b), i, workspace=ws)
    check(y, *ref.linear(x, w, a, b, None, i))
    one = layers.linear(x, w, layers.Adapters(a[2:3], b[2:3]), torch.zeros_like(i), workspace=ws)
    check(one, *ref.linear(x, w, a[2:3], b[2:3], None, torch.zeros_like(i)))


def test_adapters_index_out_of_the_stack_is_none(ws):
    g = gen(4)
    m, k, n, s, r = 40, 128, 128, 3, 8
    x, w = normal(g, "bf16", m, k), normal(g, "bf16", n, k)
    a, b, f = stack(g, "bf16", s, r, n, k)
    i = torch.tensor([-1, -5, -2 ** 31, 3, 4, 2 ** 31 - 1, 0, 1] * 5, device="cuda").int()
    y = layers.linear(x, w, layers.Adapters(a, b, f), i, workspace=ws)
    check(y, *ref.linear(x, w, a, b, f, i))
    none = i.long() > 2
    none |= i < 0
    assert torch.equal(y[none], layers.linear(x, w, workspace=ws)[none])


@pytest.mark.parametrize("s", [5, 20])  # in one launch (but pairs), and in two
@pytest.mark.parametrize("m,n", [(12, 256), (200, 256), (2048, 4096)])
def test_adapters_keep_to_their_rows(ws, m, n, s):
    """An adapter of NaN, one of infinities, rows of NaN: others' rows are as without them."""
    g = gen(5)
    k, r = 192, 16
    x, w = normal(g, "bf16", m, k), normal(g, "bf16", n, k)
    a, b, f = stack(g, "bf16", s, r, n, k)
    i = indices(g, m, 5, "own")
    clean = layers.linear(x, w, layers.Adapters(a, b, f), i, workspace=ws)
    a[1], b[2], b[3] = float("nan"), float("nan"), float("inf")
    x[4] = float("nan")
    y = layers.linear(x, w, layers.Adapters(a, b, f), i, workspace=ws)
    kept = (i == 0) | (i == 4)
    kept[4] = False
    assert kept.any()
    assert torch.equal(y[kept], clean[kept])
    assert y[4].isnan().all() and y[i == 1].isnan().all() and y[i == 2].isnan().all()
    assert not torch.isfinite(y[i == 3]).any()


def test_adapters_infinite_x(ws):
    """A row with an infinity: no NaN where the definition has none."""
    k, n, r = 64, 64, 8
    x = torch.zeros(3, k, dtype=torch.bfloat16, device="cuda")
    x[1, 5] = float("inf")
    w = torch.ones(n, k, dtype=torch.bfloat16, device="cuda")
    a = torch.ones(1, r, k, dtype=torch.bfloat16, device="cuda")
    b = torch.ones(1, n, r, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    y = layers.linear(x, w, layers.Adapters(a, b), i, workspace=ws)
    assert (y[1] == float("inf")).all() and (y[[0, 2]] == 0).all()


# ------------------------------------------------------------------ the gated product
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("m,f,k", [
    (1, 8, 8), (1, 64, 64), (1, 2816, 1024), (7, 72, 200), (16, 136, 1000), (17, 64, 65),
    (100, 1000, 328), (128, 128, 128), (333, 1000, 2200), (257, 200, 72), (1024, 1024, 512),
    (2100, 2048, 320)])
def test_gated(ws, kind, save, m, f, k):
    g = gen(m + f)
    x, w = rows16(g, kind, m, k), rows16(g, kind, 2 * f, k, k ** -0.5)
    h, hb, pre, pb = ref.gated(x, w, "silu")
    r = layers.gated(x, w, save=save, workspace=ws)
    if save:
        check(r[1], pre, pb, "pre")
        check(r[0], h, hb, "h")
    else:
        check(r, h, hb, "h")


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("m", [5, 200, 2048])
def test_gated_activations(ws, name, m):
    g = gen(m)
    x, w = normal(g, "f16", m, 128, scale=2.0), normal(g, "f16", 2048, 128, scale=128 ** -0.5)
    h, hb, _, _ = ref.gated(x, w, name)
    check(layers.gated(x, w, name, workspace=ws), h, hb)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("m", [2, 129])
def test_gated_far_values(ws, name, m):
    """Gates far out on either side, zeros, and their gradients stay finite."""
    far = torch.tensor([0.0, 1e-30, -1e-30, 30.0, -30.0, 100.0, -100.0, 1e4, -1e4, 1e18, -1e18],
                       device="cuda").bfloat16()
    k, f = 8, 16
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = far.repeat(m)[:m * len(far)].view(m, -1)[:, 0]
    x[:, 0] = far[torch.arange(m, device="cuda") % len(far)]
    w = torch.zeros(2 * f, k, dtype=torch.bfloat16, device="cuda")
    w[:f, 0], w[f:, 1], x[:, 1] = 1.0, 1.0, 0.5
    h, pre = layers.gated(x, w, name, save=True, workspace=ws)
    want, bound, wp, pb = ref.gated(x, w, name)
    check(h, want, bound + 1e-30)
    check(pre, wp, pb)
    dh = torch.ones(m, f, dtype=torch.bfloat16, device="cuda")
    dx, dw = layers.gated_backward(dh, x, w, pre, name, workspace=ws)
    grads = ref.backward(x, w, pre, name, dh=dh)
    check(dx, *grads["dx"])
    check(dw, *grads["dw_in"])


# ------------------------------------------------------------------ gradients
SIZES = [(1, 8, 8), (1, 200, 72), (7, 64, 136), (100, 328, 200), (128, 128, 128), (129, 72, 264),
         (333, 1000, 520), (777, 264, 136), (512, 2816, 1024)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,f,k", SIZES)
def test_gated_backward(ws, kind, m, f, k):
    g = gen(m + f)
    x, w = normal(g, kind, m, k), normal(g, kind, 2 * f, k, scale=k ** -0.5)
    pre, dh = normal(g, kind, m, 2 * f), normal(g, kind, m, f, scale=0.1)
    name = ACTS[(m + f) % 3]
    dx, dw = layers.gated_backward(dh, x, w, pre, name, workspace=ws)
    want = ref.backward(x, w, pre, name, dh=dh)
    check(dx, *want["dx"], what="dx")
    check(dw, *want["dw_in"], what="dw_in")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,f,k", SIZES + [(2048, 1024, 512), (100, 4096, 2048), (1, 2816, 4096),
                                           (700, 3000, 1000), (2, 136, 528), (400, 136, 72),
                                           (55, 5680, 72), (1000, 72, 1000), (130, 1800, 104)])
def test_feed_forward_backward(ws, kind, m, f, k):
    g = gen(m + f)
    x, w = normal(g, kind, m, k), normal(g, kind, 2 * f, k, scale=k ** -0.5)
    wo, dy = normal(g, kind, k, f, scale=f ** -0.5), normal(g, kind, m, k, scale=0.1)
    pre = normal(g, kind, m, 2 * f)
    name = ACTS[(m + f) % 4]
    got = layers.feed_forward_backward(dy, x, w, wo, pre, name, workspace=ws)
    want = ref.backward(x, w, pre, name, dy=dy, w_out=wo)
    for what, t in zip(("dx", "dw_in", "dw_out"), got):
        check(t, *want[what], what=what)


@pytest.mark.parametrize("m,f,k", [(20000, 8, 16), (5000, 8, 264), (3000, 520, 8), (300, 4096, 8),
                                   (130, 8, 4096), (1, 8, 8192), (128, 4096, 8)])
def test_narrow(ws, m, f, k):
    """Sizes far apart: one column of tiles, long sums of tiny results."""
    g = gen(m + k)
    x, w = normal(g, "bf16", m, k), normal(g, "bf16", 2 * f, k, scale=k ** -0.5)
    wo, dy = normal(g, "bf16", k, f, scale=f ** -0.5), normal(g, "bf16", m, k, scale=0.1)
    h, hb, pre, pb = ref.gated(x, w, "gelu")
    got, kept = layers.gated(x, w, "gelu", save=True, workspace=ws)
    check(got, h, hb, "h")
    check(kept, pre, pb, "pre")
    want = ref.backward(x, w, kept, "gelu", dy=dy, w_out=wo)
    for what, t in zip(("dx", "dw_in", "dw_out"),
                       layers.feed_forward_backward(dy, x, w, wo, kept, "gelu", workspace=ws)):
        check(t, *want[what], what=what)
    want = ref.backward(x, w, kept, "gelu", dh=got)
    for what, t in zip(("dx", "dw_in"), layers.gated_backward(got, x, w, kept, "gelu", workspace=ws)):
        check(t, *want[what], what=what)


def test_non_finite_stays_in_its_row(ws):
    """A token of infinities or NaN: other tokens' results are as without it."""
    for m, f, k in ((5, 64, 72), (300, 136, 200), (2048, 2048, 512)):
        g = gen(m)
        x, w = normal(g, "bf16", m, k), normal(g, "bf16", 2 * f, k, scale=k ** -0.5)
        wo, dy = normal(g, "bf16", k, f, scale=f ** -0.5), normal(g, "bf16", m, k)
        h, pre = layers.gated(x, w, save=True, workspace=ws)
        dx = layers.feed_forward_backward(dy, x, w, wo, pre, workspace=ws)[0]
        for bad in (float("nan"), float("inf")):
            xb, db, pb = x.clone(), dy.clone(), pre.clone()
            xb[3], db[2], pb[1, 0] = bad, bad, bad
            hb = layers.gated(xb, w, workspace=ws)
            assert torch.equal(hb[:3], h[:3]) and torch.equal(hb[4:], h[4:])
            assert not torch.isfinite(hb[3]).any()
            dxb = layers.feed_forward_backward(db, x, w, wo, pb, workspace=ws)[0]
            assert torch.equal(dxb[0], dx[0]) and torch.equal(dxb[3:], dx[3:])
            assert not torch.isfinite(dxb[1:3]).all()


def test_single_rows_and_columns(ws):
    """Tensors of one row with any stride, views of larger ones, expanded ones refused."""
    from stream_decomposition_abft_gb300.skgemm import SkgError
    g = gen(8)
    big = normal(g, "bf16", 9, 203)
    w = normal(g, "bf16", 16, 200)
    x = big[0:1, :200]
    check(layers.linear(x, w, workspace=ws), *ref.linear(x, w))
    with pytest.raises(SkgError, match="unsupported"):
        layers.linear(big[:, :200], w, workspace=ws)  # rows off 16-byte boundaries
    with pytest.raises(SkgError, match="unsupported"):
        layers.linear(big[0:1, 1:201], w, workspace=ws)
    with pytest.raises(SkgError, match="argument"):
        layers.linear(x.expand(4, 200), w, workspace=ws)
    with pytest.raises(SkgError, match="unsupported"):
        layers.gated(x, normal(g, "bf16", 24, 200), workspace=ws)  # hidden 12
    one = normal(g, "bf16", 1, 200)
    with pytest.raises(ValueError, match="index"):
        layers.linear(x, w, layers.Adapters(one.expand(1, 8, 200), w[:, :8][None]),
                      torch.zeros(1, dtype=torch.int64, device="cuda"), workspace=ws)
    with pytest.raises(ValueError, match="belongs to adapters"):
        layers.linear(x, w, index=torch.zeros(1, dtype=torch.int32, device="cuda"), workspace=ws)
    with pytest.raises(ValueError, match="tensor is wanted"):
        layers.linear(x, w, layers.Adapters(w[None, :8], w[:, :8][None]), workspace=ws)


def test_backward_strides(ws):
    g = gen(9)
    m, f, k = 140, 72, 203
    p8 = -k % 8
    x, w = normal(g, "bf16", m, k, pad=p8 + 8), normal(g, "bf16", 2 * f, k, scale=k ** -0.5, pad=p8)
    wo, dy = normal(g, "bf16", k, f, pad=24), normal(g, "bf16", m, k, pad=p8 + 16)
    pre, dh = normal(g, "bf16", m, 2 * f, pad=8), normal(g, "bf16", m, f, pad=8)
    want = ref.backward(x, w, pre, "silu", dy=dy, w_out=wo)
    for what, t in zip(("dx", "dw_in", "dw_out"),
                       layers.feed_forward_backward(dy, x, w, wo, pre, workspace=ws)):
        check(t, *want[what], what=what)
    want = ref.backward(x, w, pre, "silu", dh=dh)
    dx, dw = layers.gated_backward(dh, x, w, pre, workspace=ws)
    check(dx, *want["dx"])
    check(dw, *want["dw_in"])


@pytest.mark.parametrize("name", ACTS)
def test_gradients_against_differences(ws, name):
    """d/de of sum(y dy) along a direction, by central differences of the 64-bit definition."""
    g = gen(11)
    m, f, k = 37, 64, 72
    x, w = normal(g, "f16", m, k), normal(g, "f16", 2 * f, k, scale=k ** -0.5)
    wo, dy = normal(g, "f16", k, f, scale=f ** -0.5), normal(g, "f16", m, k)
    pre64 = x.double() @ w.double().t()
    dx, dwi, dwo = layers.feed_forward_backward(dy, x, w, wo, pre64.half(), name, workspace=ws)

    def loss(x, w, wo):
        p = x @ w.t()
        return ((ref.act(p[:, :f], name)[0] * p[:, f:]) @ wo.t() * dy.double()).sum()
    at = [t.double() for t in (x, w, wo)]
    for n, grad in enumerate((dx, dwi, dwo)):
        # Along the gradient itself; pre's rounding to fp16 moves it by some 2^-11 of its size,
        # a kink (relu) at 37 * 64 gates by less than a step's share.
        d = grad.double() / grad.double().norm()
        e = 1e-3
        plus, minus = list(at), list(at)
        plus[n], minus[n] = at[n] + e * d, at[n] - e * d
        slope = float(loss(*plus) - loss(*minus)) / (2 * e)
        assert abs(slope - float(grad.double().norm())) <= 4e-3 * float(grad.double().norm()), n


# ------------------------------------------------------------------ sizes of zero
def test_empty(ws):
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    o = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    assert layers.linear(e(0, 64), o(8, 64), workspace=ws).shape == (0, 8)
    assert layers.linear(o(4, 64), e(0, 64), workspace=ws).shape == (4, 0)
    assert (layers.linear(e(4, 0), e(8, 0), workspace=ws) == 0).all()
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert (layers.linear(e(4, 0), e(8, 0), layers.Adapters(e(2, 8, 0), o(2, 8, 8)), i,
                          workspace=ws) == 0).all()
    for ad in (layers.Adapters(e(0, 8, 64), e(0, 8, 8)), layers.Adapters(e(2, 0, 64), e(2, 8, 0))):
        assert (layers.linear(o(4, 64), o(8, 64), ad, i, workspace=ws) == 64).all()
    h, pre = layers.gated(e(4, 0), e(16, 0), save=True, workspace=ws)
    assert (h == 0).all() and (pre == 0).all() and pre.shape == (4, 16)
    assert layers.gated(e(0, 64), o(16, 64), workspace=ws).shape == (0, 8)
    assert layers.gated(o(3, 64), e(0, 64), workspace=ws).shape == (3, 0)
    dx, dwi, dwo = layers.feed_forward_backward(e(0, 64), e(0, 64), o(16, 64), o(64, 8), e(0, 16),
                                                workspace=ws)
    assert dx.shape == (0, 64) and (dwi == 0).all() and (dwo == 0).all()
    dx, dwi = layers.gated_backward(e(5, 0), o(5, 64), e(0, 64), e(5, 0), workspace=ws)
    assert (dx == 0).all() and dwi.shape == (0, 64)


# ------------------------------------------------------------------ as they are used
def block(g, kind, m, k, f, s, r):
    x, wi, wo = normal(g, kind, m, k), normal(g, kind, 2 * f, k, scale=k ** -0.5), \
        normal(g, kind, k, f, scale=f ** -0.5)
    a, b, scale = stack(g, kind, s, r, k, f)
    return x, wi, wo, layers.Adapters(a, b, scale), indices(g, m, s, "mixed")


@pytest.mark.parametrize("m", [1, 33, 300])
def test_together(ws, m):
    """A feed-forward whose second projection has adapters, then a training step's gradients."""
    g = gen(m)
    k, f = 264, 520
    x, wi, wo, ad, i = block(g, "bf16", m, k, f, 7, 16)
    h, pre = layers.gated(x, wi, "gelu_tanh", save=True, workspace=ws)
    y = layers.linear(h, wo, ad, i, workspace=ws)
    check(y, *ref.linear(h, wo, *ad, i))
    y2, pre2 = layers.feed_forward(x, wi, wo, "gelu_tanh", save=True, workspace=ws)
    assert torch.equal(pre2, pre) and torch.equal(y2, layers.linear(h, wo, workspace=ws))
    assert torch.equal(layers.feed_forward(x, wi, wo, "gelu_tanh", workspace=ws), y2)
    got = layers.feed_forward_backward(y, x, wi, wo, pre, "gelu_tanh", workspace=ws)
    want = ref.backward(x, wi, pre, "gelu_tanh", dy=y, w_out=wo)
    for what, t in zip(("dx", "dw_in", "dw_out"), got):
        check(t, *want[what], what=what)


def step(x, wi, wo, ad, i, ws):
    h, pre = layers.gated(x, wi, save=True, workspace=ws)
    y = layers.linear(h, wo, ad, i, workspace=ws)
    return (y, h, pre) + layers.feed_forward_backward(y, x, wi, wo, pre, workspace=ws)


@pytest.mark.parametrize("m", [1, 200, 1500])
def test_same_result_every_time(ws, m):
    args = block(gen(m), "bf16", m, 520, 264, 40, 32)
    first = step(*args, ws)
    for _ in range(3):
        for a, b in zip(first, step(*args, ws)):
            assert torch.equal(a, b)


def test_streams_and_graphs(ws):
    """Other streams, two captured graphs that share a workspace and run at once, and inputs that
    change between replays."""
    cases = [block(gen(n), "bf16", m, 264, 264, 9, 16) for n, m in enumerate((40, 300))]
    want = [step(*c, ws) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, c, w in zip(streams, cases, want):
        got = layers.linear(w[1], c[2], c[3], c[4], workspace=ws, stream=s)
        s.synchronize()
        assert torch.equal(got, w[0])
    graphs, outs = [], []
    for c in cases:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(step(*c, ws))
        graphs.append(gr)
    for _ in range(3):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            for a, b in zip(o, w):
                assert torch.equal(a, b)
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
    c = cases[1]
    c[0].mul_(0.5)
    c[4].copy_(c[4].flip(0).contiguous())
    graphs[1].replay()
    torch.cuda.synchronize()
    for a, b in zip(outs[1], step(*c, ws)):
        assert torch.equal(a, b)


def test_default_workspace_and_other_operators():
    """Without a workspace, behind and ahead of other kernels that the stream runs."""
    x, wi, wo, ad, i = block(gen(2), "bf16", 64, 256, 256, 4, 16)
    want = layers.linear(x, wo[:, :256], ad, i)
    for _ in range(20):
        big = torch.empty(1 << 24, device="cuda").normal_()
        x2 = (x.float() * 2).bfloat16()          # a producer just before the call
        y = layers.linear(x2, wo[:, :256], ad, i)
        q = mx.quantize(y, "mxfp8")              # a consumer just behind it
        del x2
        assert torch.equal(y, (want.float() * 2).bfloat16())
        assert torch.equal(q.codes, mx.quantize((want.float() * 2).bfloat16(), "mxfp8").codes)
        del big


def test_more_than_2_to_31_elements(ws):
    m, n, k = 40000, 57344, 64
    g = gen(6)
    x, w = normal(g, "bf16", m, k), normal(g, "bf16", n, k)
    y = layers.linear(x, w, workspace=ws)
    pick = torch.tensor([0, 1, 20000, 37449, 37450, 39998, 39999], device="cuda")
    check(y[pick], *ref.linear(x[pick], w))
    del y
    h = layers.gated(x, w, workspace=ws)
    hw, hb, _, _ = ref.gated(x[pick], w, "silu")
    check(h[pick], hw, hb)
