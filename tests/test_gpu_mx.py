"""Microscaled operators on the GPU against the 64-bit oracle.

Tolerances, derived from the formats and fp32 (u = 2^-24):
 - quantisation is defined to the bit: codes, scales and values compare equal.
 - norm: a row's sum of squares runs over at most 64 terms in a thread, a tree
   of at most 10 levels and 16 warps, each within u: rstd within 100 u relative,
   and y = h rstd w within 110 u. A code is the nearest one to y / s, so
   |value - y| <= half a step (2^-4 |y| or 2^-10 s) plus that.
 - gradient: the row's mean and the products likewise, 200 u times the sum of
   the magnitudes of dx's terms, plus the output's rounding; dw: at most rows
   terms, (rows + 8) u times the sum of magnitudes.
 - product: one fp32 rounding (of up to a whole unit, 2 u) per MMA of 32 or 64
   products, one per CTA of a split: (k / 32 + 16) 2 u times sum |a||b|, and the
   output's rounding.
"""
import numpy as np
import pytest
import torch

from oracle import mx_ref as mr
from stream_decomposition_abft_gb300 import mx, skgemm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U_OUT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
FORMATS = ("mxfp8", "mxfp4", "nvfp4")


def draw(rows, cols, dtype, seed, spread=1.0):
    """Normal values, block magnitudes spread over exp(+-spread), some zero blocks."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    x *= torch.exp(spread * torch.randn(rows, (cols + 7) // 8, generator=g)) \
        .repeat_interleave(8, 1)[:, :cols]
    x *= (torch.rand(rows, (cols + 31) // 32, generator=g) > 0.1).float() \
        .repeat_interleave(32, 1)[:, :cols]
    return x.to(TYPES[dtype])


def np32(t):
    return t.float().cpu().numpy()


def np64(t):
    return t.double().cpu().numpy()


def strided(x, pad, offset=0):
    """x inside a wider buffer, `offset` elements off its start."""
    buf = torch.full((x.shape[0], x.shape[1] + pad), 7.0, dtype=x.dtype, device="cuda")
    view = buf[:, offset:offset + x.shape[1]]
    view.copy_(x)
    return view


def check_quantized(q, want_codes, want_scales):
    got = q.codes.cpu().numpy()
    assert np.array_equal(got, mr.pack(want_codes, q.format))
    assert np.array_equal(q.scales.cpu().numpy(), mr.tile_scales(want_scales))


SIZES = [(1, 1), (1, 32), (3, 17), (5, 64), (33, 96), (128, 128), (129, 160), (40, 2200),
         (257, 515), (1, 8192), (2, 28672)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,k", SIZES)
def test_quantize(fmt, dtype, rows, k):
    for transpose in (False, True):
        x = draw(rows, k, dtype, rows * 131 + k)
        g = float(x.float().abs().max()) / 2688 + 1e-6
        gt = torch.tensor([g], device="cuda") if fmt == "nvfp4" else None
        codes, scales = mr.quantize(np32(x), fmt, np.float32(g))
        src = (x.t().contiguous() if transpose else x).cuda()
        q, v = mx.quantize(src, fmt, transpose=transpose, tensor_scale=gt, values=True)
        check_quantized(q, codes, scales)
        gv = np.float32(g) if fmt == "nvfp4" else np.float32(1)
        n = mr.BLOCK[fmt]
        full = mr.scale_values(scales, fmt).astype(np.float32)
        want = (mr.code_values(codes, fmt).astype(np.float32).reshape(rows, -1, n)
                * full[..., None] * gv).reshape(rows, -1)[:, :k]
        assert torch.equal(v.cpu(), torch.from_numpy(want).to(x.dtype))
        # Without the values, the same codes.
        q2 = mx.quantize(src, fmt, transpose=transpose, tensor_scale=gt)
        assert torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 1), (16, 8)])
def test_quantize_strides(fmt, transpose, pad, offset):
    x = draw(70, 200, "bf16", 5)
    src = strided(x.t().contiguous() if transpose else x, pad, offset)
    codes, scales = mr.quantize(np32(x), fmt)
    check_quantized(mx.quantize(src, fmt, transpose=transpose), codes, scales)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 200, 0), (130, 33, 5), (257, 515, 0),
                                           (256, 384, 0), (1000, 96, 8), (5, 2200, 1)])
def test_quantize_both(fmt, dtype, rows, cols, pad):
    # One pass, the bytes of two.
    x = strided(draw(rows, cols, dtype, rows + cols), pad)
    g = torch.tensor([0.01], device="cuda") if fmt == "nvfp4" else None
    for got, tr in zip(mx.quantize_both(x, fmt, tensor_scale=g), (False, True)):
        want = mx.quantize(x, fmt, transpose=tr, tensor_scale=g)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
        assert (got.rows, got.k) == (want.rows, want.k)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_special_values(fmt):
    # Infinities and NaN spoil their own block alone; extremes of fp32, signed
    # zeros, subnormals; exact ties.
    x = torch.zeros(8, 96)
    x[0, 5], x[0, 40] = float("inf"), 1.0
    x[1, 70], x[1, 0] = float("nan"), 2.0
    x[2, :32] = 3.4e38
    x[3, :32] = 1e-45
    x[4, :64] = -0.0
    x[5, :16] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75,
                              -2.5, -3.5, -5, -6])
    x[6, 31], x[6, 32] = float("-inf"), -1.0
    x[7, :3] = torch.tensor([1.1754943508222875e-38, -1e-39, 1e-41])
    for transpose in (False, True):
        src = (x.t().contiguous() if transpose else x).cuda()
        q, v = mx.quantize(src, fmt, transpose=transpose, values=True)
        codes, scales = mr.quantize(x.numpy(), fmt)
        check_quantized(q, codes, scales)
        nan = np.repeat(~np.isfinite(x.numpy()).reshape(8, -1, mr.BLOCK[fmt]).all(-1),
                        mr.BLOCK[fmt], 1)
        assert np.array_equal(np.isnan(v.cpu().numpy()), nan)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_large_offset(fmt):
    # Rows whose element offsets pass 2^31.
    ld, rows = 1 << 22, 516
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    view = buf.view(rows, ld)[:, :96]
    x = draw(rows, 96, "bf16", 9)
    view.copy_(x)
    assert (rows - 1) * ld > 2 ** 31
    codes, scales = mr.quantize(np32(x), fmt)
    check_quantized(mx.quantize(view, fmt), codes, scales)


def test_quantize_many_rows():
    # More rows than one grid covers: the same bytes as for their last tiles alone.
    rows, k = 1_100_000, 512
    x = torch.randn(rows, k, device="cuda", dtype=torch.bfloat16)
    q = mx.quantize(x, "mxfp8")
    first = (rows - 1000) // 128 * 128
    tail = mx.quantize(x[first:], "mxfp8")
    assert torch.equal(q.codes[first:], tail.codes)
    assert torch.equal(q.scales[first // 128 * (k // 128) * 512:], tail.scales)


# ------------------------------------------------------------------ norm
def check_norm(x, w, res, fmt, eps, g=None):
    gt = None if g is None else torch.tensor([g], device="cuda")
    q, h, rstd = mx.rmsnorm(x, w, eps, residual=res, format=fmt, tensor_scale=gt)
    rows, cols = x.shape
    y, h64, r64 = mr.rmsnorm(np64(x), np64(w), eps, None if res is None else np64(res))
    assert np.all(np.abs(np64(rstd) - r64) <= 100 * U * r64)
    if res is None:
        assert h is None
    else:
        want = (x.float() + res.float()).to(x.dtype)
        assert torch.equal(h, want)
    n = mr.BLOCK[fmt]
    nb = -(-cols // 32) * 32 // n
    groups = -(-nb // 4)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    stored = q.scales.cpu().numpy()
    sb = stored[mr.scale_offset(r, b, groups)]
    assert np.array_equal(mr.tile_scales(sb), stored)  # zeros everywhere else
    codes = mr.unpack(q.codes.cpu().numpy(), fmt)
    assert not codes[:, cols:].any()
    s = mr.scale_values(sb, fmt) * (1.0 if g is None else float(np.float32(g)))
    yb = mr.pad_k(y).reshape(rows, nb, n)
    amax = np.abs(yb).max(-1)
    tol = 110 * U
    if fmt == "nvfp4":
        gg = 1.0 if g is None else float(np.float32(g))
        t = np.minimum(amax / (6 * gg), 448)
        assert np.all(np.abs(s / gg - t) <= t * (2.0 ** -4 + tol) + 2.0 ** -10)
    else:
        most = 448.0 if fmt == "mxfp8" else 6.0
        assert np.all(amax <= most * s * (1 + tol))
        assert np.all((amax > most * s / 2 * (1 - tol)) | (sb == 0))
    v = mr.code_values(codes, fmt).reshape(rows, nb, n) * s[..., None]
    if fmt == "mxfp8":
        half = np.maximum(2.0 ** -4 * np.abs(yb), 2.0 ** -10 * s[..., None])
    else:  # steps of 1/2 below 2, 1 below 4, 2 below 6; above 6 s it saturates (nvfp4)
        a = np.abs(yb) / np.maximum(s[..., None], 1e-300)
        half = np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, 1.0)) * s[..., None]
        if fmt == "nvfp4":
            half = np.maximum(half, np.abs(yb) - 6 * s[..., None])
    assert np.all(np.abs(v - yb) <= half * (1 + 2 * tol) + tol * np.abs(yb) + 1e-300)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8192), (2, 40), (7, 128), (130, 333),
                                       (64, 2200), (3, 16384), (2, 28672), (2, 40000), (3, 12001),
                                       (2, 30001), (2, 33333)])
def test_rmsnorm(fmt, dtype, rows, cols):
    g = torch.Generator().manual_seed(cols)
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(TYPES[dtype]).cuda()
    for with_res in (False, True):
        x = draw(rows, cols, dtype, 3 * cols + rows, 0.5).cuda()
        res = draw(rows, cols, dtype, 5 * cols + rows, 0.5).cuda() if with_res else None
        check_norm(x, w, res, fmt, 1e-5, 0.003 if fmt == "nvfp4" else None)


@pytest.mark.parametrize("pad,offset", [(8, 0), (5, 3)])
def test_rmsnorm_strides_and_zero_rows(pad, offset):
    x, r = draw(37, 264, "bf16", 1), draw(37, 264, "bf16", 2)
    x[4] = 0
    r[4] = 0
    w = torch.ones(264, dtype=torch.bfloat16, device="cuda")
    check_norm(strided(x, pad, offset), w, strided(r, pad, offset), "mxfp8", 1e-6)


def test_rmsnorm_sum_in_place():
    # The sum may replace the residual (or x) itself, at any width.
    for cols in (512, 40000):
        x, r = draw(3, cols, "bf16", 1).cuda(), draw(3, cols, "bf16", 2).cuda()
        w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
        q, h, rstd = mx.rmsnorm(x, w, 1e-5, residual=r)
        codes, scales = torch.empty_like(q.codes), torch.empty_like(q.scales)
        rs = torch.empty_like(rstd)
        st = skgemm.rmsnorm_mx(3, cols, x.data_ptr(), cols, r.data_ptr(), cols, w.data_ptr(),
                               skgemm.IN_BF16, 1e-5, r.data_ptr(), cols, rs.data_ptr(),
                               skgemm.MXFP8, None, codes.data_ptr(), codes.shape[1],
                               scales.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert st == skgemm.OK
        assert torch.equal(r, h) and torch.equal(codes, q.codes) and \
            torch.equal(scales, q.scales) and torch.equal(rs, rstd)


def test_rmsnorm_nan_row_stays_alone():
    x = draw(5, 320, "bf16", 3).cuda()
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    w = torch.ones(320, dtype=torch.bfloat16, device="cuda")
    q, _, rstd = mx.rmsnorm(x, w, 1e-5)
    clean = x.clone()
    clean[2:4] = 0
    qc, _, rc = mx.rmsnorm(clean, w, 1e-5)
    keep = [0, 1, 4]
    assert torch.equal(q.codes[keep], qc.codes[keep]) and torch.equal(rstd[keep], rc[keep])
    assert bool(torch.isnan(rstd[2])) and float(rstd[3]) == 0.0
    s = q.scales.cpu().numpy()
    assert all(s[mr.scale_offset(2, b, 3)] == 0xFF for b in range(10))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8192), (5, 40), (130, 333), (333, 1111),
                                       (700, 64), (64, 2200), (9, 16384), (3, 28672), (2, 40000),
                                       (3, 12001), (2, 30001), (2, 33333)])
def test_rmsnorm_backward(dtype, rows, cols):
    g = torch.Generator().manual_seed(cols)
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(TYPES[dtype]).cuda()
    h = draw(rows, cols, dtype, cols + rows, 0.5).cuda()
    dy = draw(rows, cols, dtype, 2 * cols + rows, 0.5).cuda()
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-5)
    for dres in (None, draw(rows, cols, dtype, 7 * cols + rows, 0.5).cuda()):
        dx, dw = mx.rmsnorm_backward(dy, h, w, rstd, dresidual=dres)
        a, b, ww, r = np64(dy), np64(h), np64(w), np64(rstd)[:, None]
        want, want_w = mr.rmsnorm_backward(a, b, ww, np64(rstd),
                                           None if dres is None else np64(dres))
        xhat, u = np.abs(b * r), np.abs(a * ww)
        mag = r * (u + xhat * (u * xhat).mean(1, keepdims=True))
        if dres is not None:
            mag = mag + np.abs(np64(dres))
        u_out = U_OUT[dx.dtype]
        tiny = 2.0 ** -25 if dtype == "f16" else 0.0  # half of fp16's least step
        assert np.all(np.abs(np64(dx) - want) <= 200 * U * mag + u_out * np.abs(want) + tiny)
        assert np.all(np.abs(np64(dw) - want_w) <= (rows + 8) * U * (np.abs(a) * xhat).sum(0) * 2)
        dx2, dw2 = mx.rmsnorm_backward(dy, h, w, rstd, dresidual=dres)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("cols", [97, 1030, 4095, 5001, 8191, 8192])
@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (8, 7), (13, 4)])
def test_rmsnorm_rows_off_boundaries(cols, pad, offset):
    # Rows that start at every distance from a 16-byte boundary, forward and backward:
    # the same bits as from contiguous, aligned copies padded to the same width.
    rows = 330
    x, r, dy = (strided(draw(rows, cols, "f16", cols + i, 0.5), pad, offset) for i in range(3))
    w = strided(draw(1, cols, "f16", 9, 0.2), 1, 1)[0]
    q, h, rstd = mx.rmsnorm(x, w, 1e-5, residual=r)
    q2, h2, rstd2 = mx.rmsnorm(x.contiguous(), w.clone(), 1e-5, residual=r.contiguous())
    assert torch.equal(h, h2) and torch.equal(rstd, rstd2)
    assert torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales)
    check_norm(x[:40], w, r[:40], "mxfp8", 1e-5)
    dx, dw = mx.rmsnorm_backward(dy, x, w, rstd, dresidual=r)
    a, b, ww = np64(dy), np64(x), np64(w)
    want, want_w = mr.rmsnorm_backward(a, b, ww, np64(rstd), np64(r))
    xhat, u = np.abs(b * np64(rstd)[:, None]), np.abs(a * ww)
    mag = np64(rstd)[:, None] * (u + xhat * (u * xhat).mean(1, keepdims=True)) + np.abs(np64(r))
    assert np.all(np.abs(np64(dx) - want) <=
                  200 * U * mag + 2.0 ** -11 * np.abs(want) + 2.0 ** -25)
    assert np.all(np.abs(np64(dw) - want_w) <= (rows + 8) * U * (np.abs(a) * xhat).sum(0) * 2)


@pytest.mark.parametrize("cols", [48, 333, 1111, 8192, 12000, 40000])
@pytest.mark.parametrize("place", ["dy", "dresidual"])
def test_rmsnorm_backward_in_place(cols, place):
    # dX may take the place of dY or of the residual path's gradient.
    rows = 700 if cols < 2000 else 5
    h, dy, dr = (draw(rows, cols, "bf16", cols + i, 0.5).cuda() for i in range(3))
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-5)
    want = mx.rmsnorm_backward(dy, h, w, rstd, dresidual=dr)
    out = {"dy": dy, "dresidual": dr}[place]
    dw = torch.empty(cols, device="cuda")
    n = skgemm.workspace_size_rmsnorm_backward(rows, cols)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    st = skgemm.rmsnorm_backward(rows, cols, dy.data_ptr(), cols, h.data_ptr(), cols, w.data_ptr(),
                                 rstd.data_ptr(), dr.data_ptr(), cols, skgemm.IN_BF16,
                                 out.data_ptr(), cols, dw.data_ptr(), ws.data_ptr(), n,
                                 torch.cuda.current_stream().cuda_stream)
    assert st == skgemm.OK
    assert torch.equal(out, want[0]) and torch.equal(dw, want[1])


def test_rmsnorm_backward_against_differences():
    # Central differences of the 64-bit forward formula, through the kernel's
    # stored rstd; inputs are exact in fp16, so the formula's gradient is what
    # the kernel rounds.
    rows, cols, eps = 2, 48, 1e-3
    x, w, dy = draw(rows, cols, "f16", 1, 0.2), draw(1, cols, "f16", 2, 0.2)[0], \
        draw(rows, cols, "f16", 3, 0.2)
    _, _, rstd = mx.rmsnorm(x.cuda(), w.cuda(), eps)
    dx, dw = mx.rmsnorm_backward(dy.cuda(), x.cuda(), w.cuda(), rstd)
    X, W, D = np64(x), np64(w), np64(dy)
    loss = lambda a, b: (mr.rmsnorm(a, b, eps)[0] * D).sum()
    num_x, num_w, d = np.zeros_like(X), np.zeros_like(W), 1e-5
    for i in range(rows):
        for j in range(cols):
            e = np.zeros_like(X)
            e[i, j] = d
            num_x[i, j] = (loss(X + e, W) - loss(X - e, W)) / (2 * d)
    for j in range(cols):
        e = np.zeros_like(W)
        e[j] = d
        num_w[j] = (loss(X, W + e) - loss(X, W - e)) / (2 * d)
    # fp16 rounding (2^-11), fp32 sums, and the differences' own error.
    assert np.all(np.abs(np64(dx) - num_x) <= 2.0 ** -11 * np.abs(num_x) + 1e-5)
    assert np.all(np.abs(np64(dw) - num_w) <= 1e-5)


# ------------------------------------------------------------------ product
def operand(rows, k, fmt, seed, spread=1.0):
    x = draw(rows, k, "f32", seed, spread)
    g = np.float32(float(x.abs().max()) / 2688 + 1e-6) if fmt == "nvfp4" else np.float32(1)
    codes, scales = mr.quantize(np32(x), fmt, g)
    q = mx.Matrix(fmt, rows, k, torch.from_numpy(mr.pack(codes, fmt)).cuda(),
                  torch.from_numpy(mr.tile_scales(scales)).cuda(),
                  torch.tensor([g], device="cuda") if fmt == "nvfp4" else None)
    return q, torch.from_numpy(mr.values(codes, scales, fmt, float(g), k)).cuda()


def check_product(got, a, b, k, alpha=1.0, beta=0.0, c0=None):
    want = alpha * (a @ b.t())
    bound = abs(alpha) * (k / 32 + 16) * 2 * U * (a.abs() @ b.abs().t())
    if c0 is not None:
        want = want + beta * c0.double()
        bound = bound + 2 * U * (beta * c0.double()).abs()
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    err = (got.double() - want).abs()
    tol = bound + U_OUT[got.dtype] * want.abs() + tiny
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, worst " \
        f"{float((err / tol.clamp_min(1e-300)).nan_to_num(1e30).max()):.3g} of the tolerance"


PRODUCTS = [(1, 1, 1), (1, 128, 32), (3, 5, 7), (17, 200, 96), (128, 128, 128), (128, 256, 256),
            (129, 257, 300), (64, 1000, 2200), (16, 2048, 8192), (1, 28672, 1024), (300, 130, 1056),
            (257, 513, 544), (512, 768, 4096), (1000, 1500, 800),
            (200, 1000, 96), (100, 328, 64), (17, 88, 32), (130, 4, 32)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(fmt, m, n, k):
    a, av = operand(m, k, fmt, m + 3 * k)
    b, bv = operand(n, k, fmt, n + 5 * k)
    ws = mx.workspace()
    for dtype in TYPES.values():
        got = mx.matmul(a, b, out_dtype=dtype, workspace=ws)
        check_product(got, av, bv, k)
        assert torch.equal(got, mx.matmul(a, b, out_dtype=dtype, workspace=ws))
    rep = ws.report()
    assert rep.timeouts == 0 and rep.status_bits == 0 and rep.launches == 6


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m,n,k", [(2600, 2900, 352), (2100, 5000, 1300), (6000, 1023, 32)])
def test_product_many_tiles(fmt, m, n, k):
    # More tiles than fit the GPU at once: several per CTA, ragged at both ends.
    a, av = operand(m, k, fmt, 1)
    b, bv = operand(n, k, fmt, 2)
    ws = mx.workspace()
    for dtype in TYPES.values():
        check_product(mx.matmul(a, b, out_dtype=dtype, workspace=ws), av, bv, k)
    c0 = draw(m, n, "bf16", 3).cuda()
    out = c0.clone()
    mx.matmul(a, b, out=out, alpha=2.0, beta=-1.5, workspace=ws)
    check_product(out, av, bv, k, 2.0, -1.5, c0)
    assert ws.report().timeouts == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1)])
def test_product_alpha_beta_strides(fmt, dtype, pad, offset):
    m, n, k = 150, 203, 416
    a, av = operand(m, k, fmt, 1)
    b, bv = operand(n, k, fmt, 2)
    c0 = draw(m, n, dtype, 3).cuda()
    buf = torch.full((m, n + pad), 9.0, dtype=TYPES[dtype], device="cuda")
    out = buf[:, offset:offset + n]
    out.copy_(c0)
    mx.matmul(a, b, out=out, alpha=-0.5, beta=0.75)
    check_product(out, av, bv, k, -0.5, 0.75, c0)
    keep = [j for j in range(n + pad) if not offset <= j < offset + n]
    assert bool((buf[:, keep] == 9.0).all())
    # beta = 0 does not read C.
    out.fill_(float("nan"))
    mx.matmul(a, b, out=out)
    check_product(out, av, bv, k)


@pytest.mark.parametrize("m", [9, 200, 520])
def test_product_large_offset(m):
    # Rows of C whose element offsets pass 2^31, in each of the kernels.
    n, k, ldc = 300, 160, (1 << 31) // (m - 1) // 8 * 8 + 64
    a, av = operand(m, k, "mxfp8", 1)
    b, bv = operand(n, k, "mxfp8", 2)
    buf = torch.empty(m * ldc, dtype=torch.bfloat16, device="cuda")
    out = buf.view(m, ldc)[:, :n]
    mx.matmul(a, b, out=out)
    check_product(out, av, bv, k)


@pytest.mark.parametrize("fmt", FORMATS)
def test_product_operand_strides(fmt):
    # Codes inside wider rows (other bytes around them), k short of the pitch.
    m, n, k = 140, 90, 352
    a, av = operand(m, k, fmt, 1)
    b, bv = operand(n, k, fmt, 2)
    wide = []
    for q in (a, b):
        buf = torch.full((q.rows, q.codes.shape[1] + 48), 0xEE, dtype=torch.uint8, device="cuda")
        view = buf[:, 16:16 + q.codes.shape[1]]
        view.copy_(q.codes)
        wide.append(q._replace(codes=view))
    check_product(mx.matmul(*wide), av, bv, k)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_product_wide_scales(fmt):
    # Scales over the range where every product and sum is a normal fp32.
    m, n, k = 130, 140, 512
    a, av = operand(m, k, fmt, 1, 8.0)
    b, bv = operand(n, k, fmt, 2, 8.0)
    check_product(mx.matmul(a, b, out_dtype=torch.float32), av, bv, k)


@pytest.mark.parametrize("fmt", FORMATS)
def test_product_nan_blocks(fmt):
    # A NaN scale spoils its row of C (A's) or column (B's) and nothing else.
    m, n, k = 140, 150, 320
    a, av = operand(m, k, fmt, 1)
    b, bv = operand(n, k, fmt, 2)
    nan = 0x7F if fmt == "nvfp4" else 0xFF
    groups = -(-(k // mr.BLOCK[fmt]) // 4)
    a.scales[mr.scale_offset(131, 2, groups)] = nan
    b.scales[mr.scale_offset(7, 1, groups)] = nan
    got = mx.matmul(a, b, out_dtype=torch.float32)
    want = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    want[131], want[:, 7] = True, True
    assert torch.equal(torch.isnan(got), want)
    rows, cols = [i for i in range(m) if i != 131], [j for j in range(n) if j != 7]
    check_product(got[rows][:, cols], av[rows], bv[cols], k)


@pytest.mark.parametrize("fmt", FORMATS)
def test_product_garbage_in_padding(fmt):
    # Rows of scales past m and n (here NaN) and bytes past k do not reach C.
    m, n, k = 5, 9, 40
    a, av = operand(m, k, fmt, 1)
    b, bv = operand(n, k, fmt, 2)
    for q in (a, b):
        nb = 64 // mr.BLOCK[fmt]
        live = {mr.scale_offset(r, i, 1) for r in range(q.rows) for i in range(4)}
        assert nb <= 4
        for i in range(q.scales.numel()):
            if i not in live:
                q.scales[i] = 0x7F if fmt == "nvfp4" else 0xFF
    check_product(mx.matmul(a, b, out_dtype=torch.float32), av, bv, k)


def test_empty_sizes():
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    q = mx.quantize(x, "mxfp8")
    w = mx.quantize(torch.ones(32, 64, device="cuda"), "mxfp8")
    assert mx.matmul(q, w).shape == (0, 32)
    a, b = (mx.quantize(torch.zeros(r, 0, device="cuda"), "mxfp8") for r in (4, 3))
    c = torch.full((4, 3), 2.0, device="cuda")
    mx.matmul(a, b, out=c, beta=0.5)
    assert bool((c == 1.0).all())
    wt = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    qn, h, rstd = mx.rmsnorm(x, wt, 1e-5, residual=x)
    assert qn.rows == 0 and h.shape == (0, 64) and rstd.shape == (0,)
    dx, dw = mx.rmsnorm_backward(x, x, wt, rstd)
    assert dx.shape == (0, 64) and bool((dw == 0).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_and_gradient(fmt):
    # The layer's products are those of the quantised operands; its gradients
    # are the straight-through ones of the formula.
    m, n, k = 70, 160, 96
    x, w, dy = draw(m, k, "bf16", 1).cuda(), draw(n, k, "bf16", 2).cuda(), \
        draw(m, n, "bf16", 3).cuda()
    gs = lambda t: (t.float().abs().max() / 2688).reshape(1) if fmt == "nvfp4" else None
    ws = mx.workspace()
    qw, vw = mx.quantize(w, fmt, tensor_scale=gs(w), values=True)
    qwt, vwt = mx.quantize(w, fmt, transpose=True, tensor_scale=gs(w), values=True)
    _, vx = mx.quantize(x.float(), fmt, tensor_scale=gs(x), values=True)
    qxt, _ = mx.quantize(x, fmt, transpose=True, tensor_scale=gs(x), values=True)
    y = mx.linear(x, qw, tensor_scale=gs(x), workspace=ws)
    _, vwf = mx.quantize(w.float(), fmt, tensor_scale=gs(w), values=True)
    check_product(y, vx.double(), vwf.double(), k)
    dx, dw = mx.linear_backward(dy, qwt, qxt, tensor_scale=gs(dy), workspace=ws)
    f = lambda t, tr: mx.quantize(t.float(), fmt, transpose=tr, tensor_scale=gs(t),
                                  values=True)[1].double()
    check_product(dx, f(dy, False), f(w, True), n)
    check_product(dw, f(dy, True), f(x, True), m)


def test_other_stream():
    # Work on a stream of its own, behind and in front of other streams' work.
    s = torch.cuda.Stream()
    x = draw(300, 512, "bf16", 1).cuda()
    w = mx.quantize(draw(400, 512, "bf16", 2).cuda(), "mxfp8")
    want = mx.matmul(mx.quantize(x, "mxfp8"), w)
    torch.cuda.synchronize()
    got = [mx.matmul(mx.quantize(x, "mxfp8", stream=s), w, stream=s) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(g, want) for g in got)


def test_graph_capture():
    x = draw(40, 512, "bf16", 1).cuda()
    wt = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    w = mx.quantize(draw(384, 512, "bf16", 2).cuda(), "mxfp8")
    ws = mx.workspace()
    step = lambda: mx.matmul(mx.rmsnorm(x, wt, 1e-5, residual=x)[0], w, workspace=ws)
    want = step().clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


@pytest.mark.parametrize("fmt,bound", [("mxfp8", 0.1), ("mxfp4", 0.5), ("nvfp4", 0.4)])
def test_example_block(fmt, bound):
    # The block's outputs and gradients are off fp32 by the codes' rounding: an
    # e4m3 code is within 1/16 of its value (an e2m1 code within 1/4, or more in
    # small values), in a product of two such operands, squared between.
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "mx_block.py")
    spec = importlib.util.spec_from_file_location("mx_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    for name, err in example.run(200, 264, 520, fmt).items():
        assert err < bound, (name, err)
