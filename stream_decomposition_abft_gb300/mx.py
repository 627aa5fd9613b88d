"""Microscaled operators on torch tensors: quantisation, RMS norm with a
quantised output and its gradient, the block-scaled product, and a linear
layer made of them. All arithmetic runs in libskgemm.so's kernels (the
``skg_mx_quantize``, ``skg_rmsnorm_*`` and ``skg_gemm_mx`` entry points of
include/skgemm.h, which define the formats), reached through the compiled
binding _skg_torch (argument checks, allocation of outputs); there is no
fallback.

A training step of a linear layer y = x W^T in 8 bits::

    qx = mx.quantize(x, "mxfp8")                       # (m, k), blocks along k
    y = mx.matmul(qx, qw, workspace=ws)                # qw: (n, k)
    xt = mx.quantize(x, "mxfp8", transpose=True)       # (k, m), blocks along m
    dx, dw = mx.linear_backward(dy, qwt, xt, workspace=ws)   # qwt: W^T, (k, n)

The functions return plain tensors, without autograd history: gradients are the
calls above. The norm's weight has x's type.

Every function runs on the current stream of the tensors' device, or on
``stream``; the tensors it allocates then belong to that stream. Wrong
arguments raise ValueError, a refusal by the library SkgError.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import skgemm
from .skgemm import SkgError, Workspace

FORMATS = {"mxfp8": skgemm.MXFP8, "mxfp4": skgemm.MXFP4, "nvfp4": skgemm.NVFP4}
BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}

_binding = None


def _native():
    """The compiled binding (built in-tree by __graft_entry__.build())."""
    global _binding
    if _binding is None:
        try:
            from . import _skg_torch
        except ImportError as e:
            raise RuntimeError("_skg_torch.so is missing or does not load: build it with "
                               "__graft_entry__.build(); there is no fallback") from e
        _binding = _skg_torch
    return _binding


class Matrix(NamedTuple):
    """A quantised rows x k matrix: ``codes`` (rows, pitch) bytes, ``scales`` in
    tiles of 128 rows x 4 blocks (bytes, one dimension), and ``tensor_scale``
    (one float on the device, or None = 1). One that another program made has zero
    codes from k up to a multiple of 32 and, in 4 bits, zero scales from k up to a
    multiple of 64 (include/skgemm.h)."""
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
_defaults = {}  # device: default_workspace's


def default_workspace(device="cuda") -> Workspace:
    """The workspace of the matmul calls on a device that are given none, made on first use
    and kept: its report() shows a wait of theirs that ran out."""
    d = torch.device(device)
    if d.index is None:
        d = torch.device(d.type, torch.cuda.current_device())
    ws = _defaults.get(d)
    if ws is None:
        ws = _new_workspace(d)
        torch.cuda.current_stream(d).synchronize()  # zeroed before another stream's call
        ws = _defaults.setdefault(d, ws)
    return ws


def quantize(x, format, transpose=False, tensor_scale=None, values=False, stream=None):
    """Quantise x (rows, k), or with ``transpose`` its transpose (x: (k, rows)).

    tensor_scale: "nvfp4"'s fp32 scale, best max|x| / (448 * 6); None = 1.
    Returns a Matrix, or with ``values`` (Matrix, the values that it stands
    for, in x's dtype)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return quantize(x, format, transpose, tensor_scale, values)
    r = _native().quantize(x, format, transpose, tensor_scale, values)
    if r.__class__ is int:
        raise SkgError(r, "skg_mx_quantize")
    codes, scales, v = r
    rows, k = x.shape
    q = Matrix(format, k, rows, codes, scales, tensor_scale) if transpose else \
        Matrix(format, rows, k, codes, scales, tensor_scale)
    return (q, v) if values else q


def quantize_both(x, format, tensor_scale=None, stream=None):
    """quantize(x) and quantize(x, transpose=True) in one pass over x."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return quantize_both(x, format, tensor_scale)
    r = _native().quantize_both(x, format, tensor_scale)
    if r.__class__ is int:
        raise SkgError(r, "skg_mx_quantize_both")
    rows, cols = x.shape
    return Matrix(format, rows, cols, r[0], r[1], tensor_scale), \
        Matrix(format, cols, rows, r[2], r[3], tensor_scale)


def rmsnorm(x, weight, eps, residual=None, format="mxfp8", tensor_scale=None, stream=None):
    """h = x + residual; quantised(h / sqrt(mean(h^2) + eps) * weight).

    Returns (Matrix, h in x's dtype or None without a residual, rstd (rows,))."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rmsnorm(x, weight, eps, residual, format, tensor_scale)
    r = _native().rmsnorm(x, weight, eps, residual, format, tensor_scale)
    if r.__class__ is int:
        raise SkgError(r, "skg_rmsnorm_mx")
    codes, scales, h, rstd = r
    rows, cols = x.shape
    return Matrix(format, rows, cols, codes, scales, tensor_scale), h, rstd


def rmsnorm_backward(dy, h, weight, rstd, dresidual=None, stream=None):
    """Gradient of rmsnorm's output: (dx in dy's dtype, dweight in fp32).

    h: the sum that the norm was taken of (x itself without a residual);
    dresidual: the gradient that reaches h by another path. dx is the gradient
    of x and of the residual."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rmsnorm_backward(dy, h, weight, rstd, dresidual)
    r = _native().rmsnorm_backward(dy, h, weight, rstd, dresidual)
    if r.__class__ is int:
        raise SkgError(r, "skg_rmsnorm_backward")
    return r


def matmul(a, b, out=None, out_dtype=torch.bfloat16, alpha=1.0, beta=0.0, workspace=None,
           stream=None):
    """alpha * a b^T + beta * out of two Matrix operands (m, k) and (n, k) of one
    format; ``out`` (m, n) is written in place, or allocated in ``out_dtype``.
    workspace: mx.workspace(), kept between calls; None: default_workspace() (in a CUDA
    graph's capture before its first use: one of the graph's own, whose report is lost)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return matmul(a, b, out, out_dtype, alpha, beta, workspace)
    if workspace is None:
        d = a.codes.device
        workspace = _defaults.get(d)
        if workspace is None:
            with torch.cuda.device(d):
                capturing = torch.cuda.is_current_stream_capturing()
            workspace = _new_workspace(d) if capturing else default_workspace(d)
    r = _native().matmul(a, b, out, out_dtype, alpha, beta, workspace.buf)
    if r.__class__ is int:
        raise SkgError(r, "skg_gemm_mx")
    return r


def linear(x, w, tensor_scale=None, workspace=None, stream=None):
    """y = x W^T in w's format, in x's dtype: x (m, k) is quantised along k
    (tensor_scale: its scale, "nvfp4"), w is the Matrix (n, k)."""
    q = quantize(x, w.format, tensor_scale=tensor_scale, stream=stream)
    return matmul(q, w, out_dtype=x.dtype, workspace=workspace, stream=stream)


def linear_backward(dy, wt, xt, tensor_scale=None, workspace=None, stream=None):
    """Gradients (dx, dW) of y = x W^T in dy's dtype, each in its operand's format:
    dx = Q(dy) Q(W^T)^T and dW = Q(dy^T) Q(x^T)^T, with wt the Matrix of W^T
    (k, n) and xt the Matrix of x^T (k, m); the quantisations count as the
    identity. tensor_scale: dy's scale, "nvfp4"."""
    if wt.format == xt.format:
        rows, cols = quantize_both(dy, wt.format, tensor_scale=tensor_scale, stream=stream)
    else:
        rows = quantize(dy, wt.format, stream=stream,
                        tensor_scale=tensor_scale if wt.format == "nvfp4" else None)
        cols = quantize(dy, xt.format, transpose=True, stream=stream,
                        tensor_scale=tensor_scale if xt.format == "nvfp4" else None)
    dx = matmul(rows, wt, out_dtype=dy.dtype, workspace=workspace, stream=stream)
    dw = matmul(cols, xt, out_dtype=dy.dtype, workspace=workspace, stream=stream)
    return dx, dw
