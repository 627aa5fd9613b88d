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
``stream``; the tensors it allocates then belong to that stream. A call of a
single token takes less time on the GPU than on the host, so the checks here
read each tensor's properties once and the library is called directly.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import skgemm
from .skgemm import SkgError, Workspace

FORMATS = {"mxfp8": skgemm.MXFP8, "mxfp4": skgemm.MXFP4, "nvfp4": skgemm.NVFP4}
BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
_TYPES = {torch.float32: skgemm.OUT_F32, torch.float16: skgemm.OUT_F16,
          torch.bfloat16: skgemm.OUT_BF16}
_IN_TYPES = {torch.float16: skgemm.IN_F16, torch.bfloat16: skgemm.IN_BF16}
_F32 = {torch.float32: None}
_U8 = torch.uint8
_empty = torch.empty
# Per format, bytes of codes and blocks of 32 elements (the library's
# skg_mx_codes_ld and skg_mx_scales_size, without a call).
_LAYOUT = {"mxfp8": (32, 1), "mxfp4": (16, 1), "nvfp4": (16, 2)}


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
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _sizes(rows, k, fmt):
    """(bytes from row to row of the codes, bytes of the scales)."""
    per, nb = _LAYOUT[fmt]
    k32 = (k + 31) // 32
    return k32 * per, (rows + 127) // 128 * ((k32 * nb + 3) // 4) * 512


def _format(fmt):
    code = FORMATS.get(fmt)
    if code is None:
        raise ValueError(f"unknown format {fmt!r}: one of {', '.join(FORMATS)}")
    return code


def _matrix(name, t, types, index=None, shape=None):
    """Checks a row-major CUDA matrix; returns (rows, cols, row stride, device index)."""
    sh = t.shape
    if len(sh) != 2 or (shape is not None and sh != shape):
        want = "a matrix" if shape is None else f"a matrix of shape {tuple(shape)}"
        raise ValueError(f"{name}: {want} is wanted, got {tuple(sh)}")
    if t.dtype not in types:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is wanted")
    at = t.get_device()
    if index is not None and at != index:
        raise ValueError(f"{name}: on cuda:{at}, not on cuda:{index}")
    rows, cols = sh
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return rows, cols, (ld if rows > 1 else cols or 1), at


def _vector(name, t, n, types, index):
    """Checks a contiguous CUDA vector of n elements; returns its address."""
    if t.shape != (n,) or t.dtype not in types or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name}: a contiguous vector of {n} "
                         f"{' or '.join(map(str, types))} is wanted")
    if not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{name}: on {t.device}, not on cuda:{index}")
    return t.data_ptr()


def _scale(t, fmt, index):
    """Address of a tensor scale (None: none)."""
    if t is None:
        return None
    if fmt != "nvfp4":
        raise ValueError("tensor_scale belongs to nvfp4")
    return _scalar("tensor_scale", t, index)


def _scalar(name, t, index):
    if t.numel() != 1 or t.dtype != torch.float32 or not t.is_cuda or t.get_device() != index:
        raise ValueError(f"{name}: one float32 on cuda:{index} is wanted")
    return t.data_ptr()


class _On:
    """The device and stream of a call: entered only where they are not the
    current ones already."""

    def __init__(self, index, stream):
        self.device, self.stream = torch.cuda.device(index), torch.cuda.stream(stream)

    def __enter__(self):
        self.device.__enter__()
        self.stream.__enter__()

    def __exit__(self, *exc):
        self.stream.__exit__(*exc)
        self.device.__exit__(*exc)


def _here(index, stream):
    return stream is None and torch.cuda.current_device() == index


def quantize(x, format, transpose=False, tensor_scale=None, values=False, stream=None):
    """Quantise x (rows, k), or with ``transpose`` its transpose (x: (k, rows)).

    tensor_scale: "nvfp4"'s fp32 scale, best max|x| / (448 * 6); None = 1.
    Returns a Matrix, or with ``values`` (Matrix, the values that it stands
    for, in x's dtype)."""
    code = _format(format)
    rows, k, ldx, at = _matrix("x", x, _TYPES)
    if not _here(at, stream):
        with _On(at, stream):
            return quantize(x, format, transpose, tensor_scale, values)
    if transpose:
        rows, k = k, rows
    g = _scale(tensor_scale, format, at)
    dtype, dev = x.dtype, x.device
    ldq, nscales = _sizes(rows, k, format)
    codes = _empty((rows, ldq), dtype=_U8, device=dev)
    scales = _empty(nscales, dtype=_U8, device=dev)
    v = _empty((rows, k), dtype=dtype, device=dev) if values else None
    st = skgemm.lib().skg_mx_quantize(
        rows, k, x.data_ptr(), ldx, _TYPES[dtype], 1 if transpose else 0, code, g,
        codes.data_ptr(), ldq, scales.data_ptr(), None if v is None else v.data_ptr(), k,
        _raw_stream(at))
    if st:
        raise SkgError(st, "skg_mx_quantize")
    q = Matrix(format, rows, k, codes, scales, tensor_scale)
    return (q, v) if values else q


def rmsnorm(x, weight, eps, residual=None, format="mxfp8", tensor_scale=None, stream=None):
    """h = x + residual; quantised(h / sqrt(mean(h^2) + eps) * weight).

    Returns (Matrix, h in x's dtype or None without a residual, rstd (rows,))."""
    code = _format(format)
    rows, cols, ldx, at = _matrix("x", x, _IN_TYPES)
    if not _here(at, stream):
        with _On(at, stream):
            return rmsnorm(x, weight, eps, residual, format, tensor_scale)
    dtype, dev = x.dtype, x.device
    same = {dtype: None}
    w = _vector("weight", weight, cols, same, at)
    g = _scale(tensor_scale, format, at)
    ldq, nscales = _sizes(rows, cols, format)
    h = r = hp = None
    ldr = 0
    if residual is not None:
        ldr = _matrix("residual", residual, same, at, x.shape)[2]
        h = _empty((rows, cols), dtype=dtype, device=dev)
        r, hp = residual.data_ptr(), h.data_ptr()
    codes = _empty((rows, ldq), dtype=_U8, device=dev)
    scales = _empty(nscales, dtype=_U8, device=dev)
    rstd = _empty(rows, dtype=torch.float32, device=dev)
    st = skgemm.lib().skg_rmsnorm_mx(
        rows, cols, x.data_ptr(), ldx, r, ldr, w, _IN_TYPES[dtype], eps, hp, cols,
        rstd.data_ptr(), code, g, codes.data_ptr(), ldq, scales.data_ptr(), _raw_stream(at))
    if st:
        raise SkgError(st, "skg_rmsnorm_mx")
    return Matrix(format, rows, cols, codes, scales, tensor_scale), h, rstd


def rmsnorm_backward(dy, h, weight, rstd, dresidual=None, stream=None):
    """Gradient of rmsnorm's output: (dx in dy's dtype, dweight in fp32).

    h: the sum that the norm was taken of (x itself without a residual);
    dresidual: the gradient that reaches h by another path. dx is the gradient
    of x and of the residual."""
    rows, cols, ldy, at = _matrix("dy", dy, _IN_TYPES)
    if not _here(at, stream):
        with _On(at, stream):
            return rmsnorm_backward(dy, h, weight, rstd, dresidual)
    dtype, dev, shape = dy.dtype, dy.device, dy.shape
    same = {dtype: None}
    ldh = _matrix("h", h, same, at, shape)[2]
    w = _vector("weight", weight, cols, same, at)
    rp = _vector("rstd", rstd, rows, _F32, at)
    ldr, dr = 0, None
    if dresidual is not None:
        ldr, dr = _matrix("dresidual", dresidual, same, at, shape)[2], dresidual.data_ptr()
    L = skgemm.lib()
    nbytes = L.skg_workspace_size_rmsnorm_backward(rows, cols)
    dx = _empty((rows, cols), dtype=dtype, device=dev)
    dw = _empty(cols, dtype=torch.float32, device=dev)
    ws = _empty(nbytes, dtype=_U8, device=dev)
    st = L.skg_rmsnorm_backward(
        rows, cols, dy.data_ptr(), ldy, h.data_ptr(), ldh, w, rp, dr, ldr, _IN_TYPES[dtype],
        dx.data_ptr(), cols, dw.data_ptr(), ws.data_ptr(), nbytes, _raw_stream(at))
    if st:
        raise SkgError(st, "skg_rmsnorm_backward")
    return dx, dw


def _operand(name, q, fmt, index):
    """Checks a Matrix of format fmt; returns (row stride, address of its tensor
    scale or None, device index)."""
    if q.format != fmt:
        raise ValueError(f"{name}: {q.format}, the other operand is {fmt}")
    _format(fmt)
    c, s = q.codes, q.scales
    rows, k = q.rows, q.k
    ldq, nscales = _sizes(rows, k, fmt)
    sh = c.shape
    if c.dtype != _U8 or s.dtype != _U8 or len(sh) != 2 or sh[0] != rows or sh[1] < ldq or \
            not c.is_cuda or not s.is_cuda or not s.is_contiguous() or s.numel() < nscales:
        raise ValueError(f"{name}: codes or scales are not those of a {rows} x {k} {fmt} matrix "
                         f"on a CUDA device")
    ld, unit = c.stride()
    if unit != 1 and sh[1] > 1:
        raise ValueError(f"{name}: the codes of a row must be contiguous")
    at = c.get_device()
    if s.get_device() != at or (index is not None and at != index):
        raise ValueError(f"{name}: codes and scales are not on one device with the other operand")
    t = q.tensor_scale
    return (ld if rows > 1 else sh[1]), \
        (None if t is None else _scalar(f"{name}.tensor_scale", t, at)), at


def matmul(a, b, out=None, out_dtype=torch.bfloat16, alpha=1.0, beta=0.0, workspace=None,
           stream=None):
    """alpha * a b^T + beta * out of two Matrix operands (m, k) and (n, k) of one
    format; ``out`` (m, n) is written in place, or allocated in ``out_dtype``.
    workspace: mx.workspace(), kept between calls; None allocates one."""
    fmt = a.format
    lda, ga, at = _operand("a", a, fmt, None)
    if not _here(at, stream):
        with _On(at, stream):
            return matmul(a, b, out, out_dtype, alpha, beta, workspace)
    ldb, gb, _ = _operand("b", b, fmt, at)
    m, n, k = a.rows, b.rows, a.k
    if b.k != k:
        raise ValueError(f"a has rows of {k} elements, b of {b.k}")
    if out is None:
        if beta != 0.0:
            raise ValueError("beta is for a given out")
        if out_dtype not in _TYPES:
            raise ValueError(f"unsupported out_dtype {out_dtype}")
        out = _empty((m, n), dtype=out_dtype, device=a.codes.device)
        ldc = n
    else:
        ldc = _matrix("out", out, _TYPES, at, (m, n))[2]
        out_dtype = out.dtype
    if workspace is None:
        workspace = _new_workspace(a.codes.device)
    st = skgemm.lib().skg_gemm_mx(
        m, n, k, alpha, a.codes.data_ptr(), lda, a.scales.data_ptr(), ga, b.codes.data_ptr(), ldb,
        b.scales.data_ptr(), gb, beta, out.data_ptr(), ldc, FORMATS[fmt], _TYPES[out_dtype],
        workspace.ptr, workspace.nbytes, _raw_stream(at))
    if st:
        raise SkgError(st, "skg_gemm_mx")
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
