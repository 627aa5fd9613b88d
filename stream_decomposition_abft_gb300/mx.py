"""Microscaled operators on torch tensors: quantisation, RMS norm with a
quantised output and its gradient, the block-scaled product, and a linear
layer made of them. All arithmetic runs in libskgemm.so's kernels (the
``skg_mx_quantize``, ``skg_rmsnorm_*`` and ``skg_gemm_mx`` entry points of
include/skgemm.h, which define the formats); there is no fallback.

A training step of a linear layer y = x W^T in 8 bits::

    qx = mx.quantize(x, "mxfp8")                       # (m, k), blocks along k
    y = mx.matmul(qx, qw, workspace=ws)                # qw: (n, k)
    xt = mx.quantize(x, "mxfp8", transpose=True)       # (k, m), blocks along m
    dx, dw = mx.linear_backward(dy, qwt, xt, workspace=ws)   # qwt: W^T, (k, n)

Every function runs on the current stream of the tensors' device, or on
``stream``; the tensors it allocates then belong to that stream.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import skgemm
from .skgemm import OK, SkgError, Workspace

FORMATS = {"mxfp8": skgemm.MXFP8, "mxfp4": skgemm.MXFP4, "nvfp4": skgemm.NVFP4}
BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
_TYPES = {torch.float32: skgemm.OUT_F32, torch.float16: skgemm.OUT_F16,
          torch.bfloat16: skgemm.OUT_BF16}
_IN_TYPES = {torch.float16: skgemm.IN_F16, torch.bfloat16: skgemm.IN_BF16}


class Matrix(NamedTuple):
    """A quantised rows x k matrix: ``codes`` (rows, pitch) bytes, ``scales`` in
    tiles of 128 rows x 4 blocks (bytes, one dimension), and ``tensor_scale``
    (one float on the device, or None = 1)."""
    format: str
    rows: int
    k: int
    codes: torch.Tensor
    scales: torch.Tensor
    tensor_scale: Optional[torch.Tensor] = None


def workspace(device="cuda") -> Workspace:
    """A workspace for matmul (any sizes): the report of its device-side waits."""
    return Workspace(skgemm.workspace_size_mx(1, 1, 1, skgemm.MXFP8), device)


_new_workspace = workspace


def _handle(t, stream):
    return (torch.cuda.current_stream(t.device) if stream is None else stream).cuda_stream


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _format(fmt):
    if fmt not in FORMATS:
        raise ValueError(f"unknown format {fmt!r}: one of {', '.join(FORMATS)}")
    return FORMATS[fmt]


def _rows_of(name, t, shape=None, dtypes=_IN_TYPES):
    """Checks a row-major matrix; returns its row stride."""
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name}: a matrix{'' if shape is None else f' of shape {tuple(shape)}'} "
                         f"is wanted, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is wanted")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return t.stride(0) if rows > 1 else max(cols, 1)


def _same_device(t, **others):
    for name, o in others.items():
        if o is not None and o.device != t.device:
            raise ValueError(f"{name}: on {o.device}, not on {t.device}")


def _scalar(name, t):
    if t is None:
        return None
    if t.numel() != 1 or t.dtype != torch.float32 or not t.is_cuda:
        raise ValueError(f"{name}: one float32 on the device is wanted")
    return t.data_ptr()


def _check(st, what):
    if st != OK:
        raise SkgError(st, what)


def _new(fmt, code, rows, k, g, device, stream):
    ldq = skgemm.mx_codes_ld(k, code)
    return Matrix(fmt, rows, k, _empty((rows, ldq), torch.uint8, device, stream),
                  _empty((skgemm.mx_scales_size(rows, k, code),), torch.uint8, device, stream), g)


def quantize(x, format, transpose=False, tensor_scale=None, values=False, stream=None):
    """Quantise x (rows, k), or with ``transpose`` its transpose (x: (k, rows)).

    tensor_scale: "nvfp4"'s fp32 scale, best max|x| / (448 * 6); None = 1.
    Returns a Matrix, or with ``values`` (Matrix, the values that it stands
    for, in x's dtype)."""
    code = _format(format)
    ldx = _rows_of("x", x, None, _TYPES)
    rows, k = (x.shape[1], x.shape[0]) if transpose else x.shape
    _same_device(x, tensor_scale=tensor_scale)
    g = _scalar("tensor_scale", tensor_scale)
    if g is not None and format != "nvfp4":
        raise ValueError("tensor_scale belongs to nvfp4")
    with torch.cuda.device(x.device):
        q = _new(format, code, rows, k, tensor_scale, x.device, stream)
        v = _empty((rows, k), x.dtype, x.device, stream) if values else None
        _check(skgemm.mx_quantize(rows, k, x.data_ptr(), ldx, _TYPES[x.dtype], int(transpose), code,
                                  g, q.codes.data_ptr(), q.codes.shape[1], q.scales.data_ptr(),
                                  None if v is None else v.data_ptr(), k, _handle(x, stream)),
               "skg_mx_quantize")
    return (q, v) if values else q


def rmsnorm(x, weight, eps, residual=None, format="mxfp8", tensor_scale=None, stream=None):
    """h = x + residual; quantised(h / sqrt(mean(h^2) + eps) * weight).

    Returns (Matrix, h in x's dtype or None without a residual, rstd (rows,))."""
    code = _format(format)
    ldx = _rows_of("x", x)
    rows, cols = x.shape
    ldr = _rows_of("residual", residual, x.shape, (x.dtype,)) if residual is not None else 0
    if tuple(weight.shape) != (cols,) or weight.dtype != x.dtype or \
            (cols > 1 and weight.stride(0) != 1):
        raise ValueError(f"weight: a contiguous vector of {cols} {x.dtype} is wanted")
    _same_device(x, weight=weight, residual=residual, tensor_scale=tensor_scale)
    g = _scalar("tensor_scale", tensor_scale)
    if g is not None and format != "nvfp4":
        raise ValueError("tensor_scale belongs to nvfp4")
    with torch.cuda.device(x.device):
        q = _new(format, code, rows, cols, tensor_scale, x.device, stream)
        h = None if residual is None else _empty((rows, cols), x.dtype, x.device, stream)
        rstd = _empty((rows,), torch.float32, x.device, stream)
        _check(skgemm.rmsnorm_mx(
            rows, cols, x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr,
            weight.data_ptr(), _IN_TYPES[x.dtype], eps, None if h is None else h.data_ptr(), cols,
            rstd.data_ptr(), code, g, q.codes.data_ptr(), q.codes.shape[1], q.scales.data_ptr(),
            _handle(x, stream)), "skg_rmsnorm_mx")
    return q, h, rstd


def rmsnorm_backward(dy, h, weight, rstd, dresidual=None, stream=None):
    """Gradient of rmsnorm's output: (dx in dy's dtype, dweight in fp32).

    h: the sum that the norm was taken of (x itself without a residual);
    dresidual: the gradient that reaches h by another path. dx is the gradient
    of x and of the residual."""
    ldy = _rows_of("dy", dy)
    rows, cols = dy.shape
    ldh = _rows_of("h", h, dy.shape, (dy.dtype,))
    ldr = _rows_of("dresidual", dresidual, dy.shape, (dy.dtype,)) if dresidual is not None else 0
    if tuple(weight.shape) != (cols,) or weight.dtype != dy.dtype or \
            (cols > 1 and weight.stride(0) != 1):
        raise ValueError(f"weight: a contiguous vector of {cols} {dy.dtype} is wanted")
    if tuple(rstd.shape) != (rows,) or rstd.dtype != torch.float32 or \
            (rows > 1 and rstd.stride(0) != 1):
        raise ValueError(f"rstd: a contiguous vector of {rows} float32 is wanted")
    _same_device(dy, h=h, weight=weight, rstd=rstd, dresidual=dresidual)
    with torch.cuda.device(dy.device):
        dx = _empty((rows, cols), dy.dtype, dy.device, stream)
        dw = _empty((cols,), torch.float32, dy.device, stream)
        nbytes = skgemm.workspace_size_rmsnorm_backward(rows, cols)
        ws = _empty((nbytes,), torch.uint8, dy.device, stream)
        _check(skgemm.rmsnorm_backward(
            rows, cols, dy.data_ptr(), ldy, h.data_ptr(), ldh, weight.data_ptr(), rstd.data_ptr(),
            None if dresidual is None else dresidual.data_ptr(), ldr, _IN_TYPES[dy.dtype],
            dx.data_ptr(), cols, dw.data_ptr(), ws.data_ptr(), nbytes, _handle(dy, stream)),
            "skg_rmsnorm_backward")
    return dx, dw


def _operand(name, q, fmt, device):
    code = _format(q.format)
    if q.format != fmt:
        raise ValueError(f"{name}: {q.format}, the other operand is {fmt}")
    c, s = q.codes, q.scales
    if c.dtype != torch.uint8 or s.dtype != torch.uint8 or not c.is_cuda or c.dim() != 2 or \
            c.shape[0] != q.rows or c.shape[1] < skgemm.mx_codes_ld(q.k, code) or \
            (c.shape[1] > 1 and c.stride(1) != 1) or not s.is_contiguous() or \
            s.numel() < skgemm.mx_scales_size(q.rows, q.k, code):
        raise ValueError(f"{name}: codes or scales are not those of a {q.rows} x {q.k} "
                         f"{q.format} matrix")
    _same_device(c, **{f"{name}.scales": s, f"{name}.tensor_scale": q.tensor_scale})
    if c.device != device:
        raise ValueError(f"{name}: on {c.device}, not on {device}")
    return c.stride(0) if q.rows > 1 else c.shape[1], _scalar(f"{name}.tensor_scale", q.tensor_scale)


def matmul(a, b, out=None, out_dtype=torch.bfloat16, alpha=1.0, beta=0.0, workspace=None,
           stream=None):
    """alpha * a b^T + beta * out of two Matrix operands (m, k) and (n, k) of one
    format; ``out`` (m, n) is written in place, or allocated in ``out_dtype``.
    workspace: mx.workspace(), kept between calls; None allocates one."""
    device = a.codes.device
    lda, ga = _operand("a", a, a.format, device)
    ldb, gb = _operand("b", b, a.format, device)
    if a.k != b.k:
        raise ValueError(f"a has rows of {a.k} elements, b of {b.k}")
    m, n, k = a.rows, b.rows, a.k
    with torch.cuda.device(device):
        if out is None:
            if beta != 0.0:
                raise ValueError("beta is for a given out")
            if out_dtype not in _TYPES:
                raise ValueError(f"unsupported out_dtype {out_dtype}")
            out = _empty((m, n), out_dtype, device, stream)
            ldc = n
        else:
            ldc = _rows_of("out", out, (m, n), _TYPES)
            _same_device(a.codes, out=out)
        if workspace is None:
            with torch.cuda.stream(stream):  # None: the current one
                workspace = _new_workspace(device)
        _check(skgemm.gemm_mx(m, n, k, alpha, a.codes.data_ptr(), lda, a.scales.data_ptr(), ga,
                              b.codes.data_ptr(), ldb, b.scales.data_ptr(), gb, beta,
                              out.data_ptr(), ldc, FORMATS[a.format], _TYPES[out.dtype],
                              workspace.ptr, workspace.nbytes, _handle(a.codes, stream)),
               "skg_gemm_mx")
    return out


def linear(x, w, tensor_scale=None, workspace=None, stream=None):
    """y = x W^T in w's format, in x's dtype: x (m, k) is quantised along k
    (tensor_scale: its scale, "nvfp4"), w is the Matrix (n, k)."""
    q = quantize(x, w.format, tensor_scale=tensor_scale, stream=stream)
    return matmul(q, w, out_dtype=x.dtype, workspace=workspace, stream=stream)


def linear_backward(dy, wt, xt, tensor_scale=None, workspace=None, stream=None):
    """Gradients (dx, dW) of y = x W^T in dy's dtype, in one format:
    dx = Q(dy) Q(W^T)^T and dW = Q(dy^T) Q(x^T)^T, with wt the Matrix of W^T
    (k, n) and xt the Matrix of x^T (k, m); the quantisations count as the
    identity. tensor_scale: dy's scale, "nvfp4"."""
    rows = quantize(dy, wt.format, tensor_scale=tensor_scale, stream=stream)
    cols = quantize(dy, xt.format, transpose=True, tensor_scale=tensor_scale, stream=stream)
    dx = matmul(rows, wt, out_dtype=dy.dtype, workspace=workspace, stream=stream)
    dw = matmul(cols, xt, out_dtype=dy.dtype, workspace=workspace, stream=stream)
    return dx, dw
