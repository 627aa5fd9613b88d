"""The microscaled operators' pipelined kernels with many rows or tiles to a block, so that
their rings of shared memory wrap around: each row's result is that of the row run among
few others (a block then takes one row, and no stage is used twice), bit by bit.

Tolerances, with u = 2^-24, t the terms that a thread adds in turn and a tree of at most
10 levels behind them:
 - rstd: the squares within 3 u, their sum within (t + 10) u, of which the root takes half,
   and two roundings of its own: (t / 2 + 10) u.
 - dw: a block adds its rows in turn (at most rows / SMs, rounded up), the reduction 5
   partials in turn behind two and five levels; a term takes three roundings:
   (rows / SMs + 20) u times the sum of magnitudes. One row left out is some hundred
   times that.
"""
import numpy as np
import pytest
import torch

from oracle import mx_ref as mr
from stream_decomposition_abft_gb300 import mx, skgemm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def normal(rows, cols, dtype, seed, pad=0):
    """Normal values, in rows of cols + pad elements."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g, device="cuda").to(DTYPES[dtype])
    return x[:, :cols]


def weight(cols, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(DTYPES[dtype])


def stream():
    return torch.cuda.current_stream().cuda_stream


def norm_into(x, w, res, sum_, fmt="mxfp8"):
    """The C entry, with the sum wherever the caller wants it: (codes, scales, rstd)."""
    rows, cols = x.shape
    f = mx.FORMATS[fmt]
    ldq = skgemm.mx_codes_ld(cols, f)
    codes = torch.empty(rows, ldq, dtype=torch.uint8, device="cuda")
    scales = torch.empty(skgemm.mx_scales_size(rows, cols, f), dtype=torch.uint8, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    st = skgemm.rmsnorm_mx(rows, cols, x.data_ptr(), x.stride(0), res.data_ptr(), res.stride(0),
                           w.data_ptr(), skgemm.IN_BF16 if x.dtype == torch.bfloat16 else
                           skgemm.IN_F16, EPS, sum_.data_ptr(), sum_.stride(0), rstd.data_ptr(), f,
                           None, codes.data_ptr(), ldq, scales.data_ptr(), stream())
    assert st == skgemm.OK
    return codes, scales, rstd


# (rows, columns, elements between rows): six rows or more to a block of each launch.
NORMS = [(2500, 8192, 0), (2500, 8191, 0), (2500, 8191, 9), (2600, 4095, 0), (2600, 4096, 8),
         (2600, 6000, 3), (5000, 2048, 0), (3100, 2047, 0), (8000, 1030, 0), (9000, 800, 0)]


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("rows,cols,pad", NORMS)
def test_norm_of_many_rows(fmt, rows, cols, pad):
    x, r = normal(rows, cols, "bf16", 1, pad), normal(rows, cols, "bf16", 2, pad)
    w = weight(cols, "bf16", 3)
    q, h, rstd = mx.rmsnorm(x, w, EPS, residual=r, format=fmt)
    assert torch.equal(h, (x.float() + r.float()).bfloat16())
    want = 1 / torch.sqrt((x.double() + r.double()).square().mean(1) + EPS)
    assert bool(((rstd.double() - want).abs() <= (16 / 2 + 10) * U * want).all())
    for i in range(0, rows, 128):  # 128 rows of scales are a tile of their own
        q1, h1, rstd1 = mx.rmsnorm(x[i:i + 128], w, EPS, residual=r[i:i + 128], format=fmt)
        n = q1.scales.numel()
        at = i // 128 * (q.scales.numel() // -(-rows // 128))
        assert torch.equal(q.codes[i:i + 128], q1.codes)
        assert torch.equal(q.scales[at:at + n], q1.scales)
        assert torch.equal(h[i:i + 128], h1) and torch.equal(rstd[i:i + 128], rstd1)


@pytest.mark.parametrize("place", ["x", "residual"])
@pytest.mark.parametrize("rows,cols,pad", NORMS)
def test_norm_sum_in_place_of_many_rows(rows, cols, pad, place):
    # Later rows are fetched while the sum of earlier ones is written over them.
    x, r = normal(rows, cols, "f16", 4, pad), normal(rows, cols, "f16", 5, pad)
    w = weight(cols, "f16", 6)
    want = torch.empty(rows, cols, dtype=x.dtype, device="cuda")
    outer = norm_into(x, w, r, want)
    assert torch.equal(want, (x.float() + r.float()).half())
    over = {"x": x, "residual": r}[place]
    inner = norm_into(x, w, r, over)
    assert torch.equal(over, want)
    assert all(torch.equal(a, b) for a, b in zip(inner, outer))


@pytest.mark.parametrize("with_res", [False, True])
@pytest.mark.parametrize("rows,cols,pad", [(1600, 8192, 0), (1600, 8191, 0), (1600, 5001, 0),
                                           (1600, 5000, 3), (1600, 4096, 0), (1600, 4095, 1),
                                           (4500, 1030, 0), (4500, 2048, 0), (5500, 512, 0),
                                           (5500, 511, 0)])
def test_norm_gradient_of_many_rows(rows, cols, pad, with_res):
    h, dy = normal(rows, cols, "bf16", 1, pad), normal(rows, cols, "bf16", 2, pad)
    dr = normal(rows, cols, "bf16", 3, pad) if with_res else None
    w = weight(cols, "bf16", 4)
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    dx, dw = mx.rmsnorm_backward(dy, h, w, rstd, dresidual=dr)
    xhat = h.double() * rstd.double()[:, None]
    terms = dy.double() * xhat
    n = -(-rows // skgemm.device_sm_count())
    assert bool(((dw.double() - terms.sum(0)).abs() <= (n + 20) * U * terms.abs().sum(0)).all())
    for i in range(0, rows, 150):  # a block each
        d1, _ = mx.rmsnorm_backward(dy[i:i + 150], h[i:i + 150], w, rstd[i:i + 150],
                                    dresidual=None if dr is None else dr[i:i + 150])
        assert torch.equal(dx[i:i + 150], d1), i
    # In place of dY: later rows of it are fetched while dX is written.
    nb = skgemm.workspace_size_rmsnorm_backward(rows, cols)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    dw2 = torch.empty(cols, device="cuda")
    st = skgemm.rmsnorm_backward(rows, cols, dy.data_ptr(), dy.stride(0), h.data_ptr(),
                                 h.stride(0), w.data_ptr(), rstd.data_ptr(),
                                 dr.data_ptr() if with_res else None,
                                 dr.stride(0) if with_res else 0, skgemm.IN_BF16, dy.data_ptr(),
                                 dy.stride(0), dw2.data_ptr(), ws.data_ptr(), nb, stream())
    assert st == skgemm.OK
    assert torch.equal(dy, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(5000, 5001), (5000, 5008), (5001, 5003)])
def test_quantize_columns_of_many_tiles(fmt, dtype, rows, cols):
    # Several tiles to a block: the bytes that the row kernel writes of the transpose,
    # and the oracle's for the last rows of it.
    x = normal(rows, cols, dtype, 7)
    g = torch.tensor([0.004], device="cuda") if fmt == "nvfp4" else None
    want, values = mx.quantize(x.t().contiguous(), fmt, tensor_scale=g, values=True)
    got, got_values = mx.quantize(x, fmt, transpose=True, tensor_scale=g, values=True)
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    assert torch.equal(got_values, values)
    row, col = mx.quantize_both(x, fmt, tensor_scale=g)
    assert torch.equal(col.codes, want.codes) and torch.equal(col.scales, want.scales)
    along = mx.quantize(x, fmt, tensor_scale=g)
    assert torch.equal(row.codes, along.codes) and torch.equal(row.scales, along.scales)
    codes, _ = mr.quantize(x[:, -3:].t().float().cpu().numpy(), fmt,
                           np.float32(0.004) if fmt == "nvfp4" else 1.0)
    assert np.array_equal(got.codes[-3:].cpu().numpy(), mr.pack(codes, fmt))


@pytest.mark.parametrize("cols,pad", [(4096, 3), (8192, 5), (2048, 1), (800, 7), (264, 2)])
def test_norm_off_boundaries_against_aligned(cols, pad):
    # Rows off 16-byte boundaries against copies on them: other kernels, the same bits in
    # the sum; statistics within their tolerance (their terms are added in the same order).
    rows = 700
    x, r, dy = (normal(rows, cols, "bf16", i, pad) for i in (1, 2, 3))
    assert x.stride(0) % 8
    w = weight(cols, "bf16", 4)
    q, h, rstd = mx.rmsnorm(x, w, EPS, residual=r)
    q2, h2, rstd2 = mx.rmsnorm(x.contiguous(), w, EPS, residual=r.contiguous())
    assert torch.equal(h, h2)
    assert bool(((rstd - rstd2).double().abs() <= 2 * (16 / 2 + 10) * U * rstd2).all())
    # A code differs only where its value falls on a tie's two sides: with steps of 1/16 of
    # the value or more, for at most 16 times the statistics' difference of them.
    assert float((q.codes != q2.codes).float().mean()) <= 16 * 2 * (16 / 2 + 12) * U
    dx, dw = mx.rmsnorm_backward(dy, x, w, rstd, dresidual=r)
    dx2, dw2 = mx.rmsnorm_backward(dy.contiguous(), x.contiguous(), w, rstd,
                                   dresidual=r.contiguous())
    xhat, u = (x.double() * rstd[:, None]).abs(), (dy.double() * w).abs()
    mag = rstd.double()[:, None] * (u + xhat * (u * xhat).mean(1, keepdim=True)) + r.double().abs()
    # Two roundings to bf16, which may fall to either side.
    most = torch.maximum(dx.abs(), dx2.abs()).double()
    assert bool(((dx.double() - dx2.double()).abs() <= 400 * U * mag + 2.0 ** -7 * most).all())
    mag = (dy.double().abs() * xhat).sum(0)
    n = -(-rows // skgemm.device_sm_count())
    assert bool(((dw.double() - dw2.double()).abs() <= 2 * (n + 20) * U * mag).all())
