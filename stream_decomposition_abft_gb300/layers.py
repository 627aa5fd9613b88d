"""A layer's projections in 16 bits on torch tensors: the gated feed-forward (both
projections, the activation and the product in one kernel) with its gradients, and a
projection with the low-rank adapters of many requests beside it. All arithmetic
runs in libskgemm.so's kernels (the ``skg_linear``, ``skg_gated``,
``skg_gated_backward`` and ``skg_feed_forward_backward`` entry points of
include/skgemm.h), reached through the compiled binding _skg_torch; there is no
fallback.

Serving, every row with the adapter of its request::

    adapters = layers.Adapters(down, up, scale)        # (S, r, k), (S, n, r), (S,)
    y = layers.linear(x, w, adapters, index, workspace=ws)   # index: int32 per row, -1: none

A training step of a feed-forward y = (act(x W_gate^T) * (x W_up^T)) W_out^T, with
w_in = [W_gate; W_up] (2 hidden, k)::

    y, pre = layers.feed_forward(x, w_in, w_out, "silu", save=True, workspace=ws)
    dx, dw_in, dw_out = layers.feed_forward_backward(dy, x, w_in, w_out, pre, "silu",
                                                     workspace=ws)

Tensors are fp16 or bf16, all of one type, with a contiguous last dimension, rows on
16-byte boundaries, and a hidden size that is a multiple of 8. The functions return
plain tensors, without autograd history, whether or not their inputs require a gradient:
gradients are the calls above. Adapters are for serving: they have no gradient here.

Between the gradients' products the projections' gradients (and act(gate) * up, formed
again) are rounded to the tensors' type, from 129 rows on once, up to 128 rows to twice
its mantissa. In fp16 they have its range: zero below 2^-25, infinite beyond 65504, so
losses are scaled as in any fp16 training. An infinite weight gives infinities or NaN in
the results that it reaches, not always the one that the formula has.

Every function runs on the current stream of the tensors' device, or on ``stream``;
the tensors it allocates then belong to that stream. ``workspace``:
``layers.workspace()``, kept between calls (it may serve several streams); None:
``mx.default_workspace()``'s rule. Wrong arguments raise ValueError, a refusal by the
library SkgError.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import mx, skgemm
from .skgemm import SkgError, Workspace

ACTIVATIONS = {"silu": skgemm.ACT_SILU, "gelu": skgemm.ACT_GELU,
               "gelu_tanh": skgemm.ACT_GELU_TANH, "relu": skgemm.ACT_RELU}


class Adapters(NamedTuple):
    """A stack of low-rank adapters of one projection: ``down`` (S, rank, k), ``up``
    (S, n, rank) and ``scale`` (S,) in fp32 (None: 1). Ranks are multiples of 8, at
    most 512; smaller adapters fill their rest with zeros."""
    down: torch.Tensor
    up: torch.Tensor
    scale: Optional[torch.Tensor] = None


def workspace(device="cuda") -> Workspace:
    """A workspace for the calls of this module (any sizes): the report of their
    device-side waits."""
    return Workspace(skgemm.workspace_size_layers(), device)


def _buffer(ws, x):
    """The workspace's buffer; without one the device's default (mx.matmul's rule)."""
    if ws is None:
        d = x.device if isinstance(x, torch.Tensor) else None
        if d is None or d.type != "cuda":
            raise ValueError("x: a CUDA tensor is wanted")
        ws = mx.workspace_for(d)
    return ws.buf


def linear(x, w, adapters=None, index=None, out=None, workspace=None, stream=None):
    """y = x w^T, and with ``adapters`` y_i += scale_s (x_i down_s^T) up_s^T for every row
    with adapter s = index[i].

    x (m, k), w (n, k); index: (m,) int32 on the device, in any order, a value that is
    negative or not below S for none. ``out`` (m, n) is written in place (it shares no memory
    with an input: refused), or allocated (for n that is no multiple of 8 as a view of padded
    rows)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear(x, w, adapters, index, out, workspace)
    r = mx._native().linear(x, w, adapters, index, out, _buffer(workspace, x))
    if r.__class__ is int:
        raise SkgError(r, "skg_linear")
    return r


def gated(x, w_in, activation="silu", save=False, workspace=None, stream=None):
    """h = act(x W_gate^T) * (x W_up^T), w_in = [W_gate; W_up] (2 hidden, k).

    Returns h (m, hidden), or with ``save`` (h, pre): pre (m, 2 hidden) is x w_in^T, which
    the gradients want."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated(x, w_in, activation, save, workspace)
    r = mx._native().gated(x, w_in, activation, save, _buffer(workspace, x))
    if r.__class__ is int:
        raise SkgError(r, "skg_gated")
    return r if save else r[0]


def gated_backward(dh, x, w_in, pre, activation="silu", workspace=None, stream=None):
    """Gradients (dx, dw_in) of gated from dh (m, hidden)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated_backward(dh, x, w_in, pre, activation, workspace)
    r = mx._native().gated_backward(dh, x, w_in, pre, activation, _buffer(workspace, x))
    if r.__class__ is int:
        raise SkgError(r, "skg_gated_backward")
    return r


def feed_forward(x, w_in, w_out, activation="silu", save=False, workspace=None, stream=None):
    """y = gated(x, w_in) w_out^T (w_out: (k, hidden)); with ``save`` (y, pre)."""
    r = gated(x, w_in, activation, save, workspace, stream)
    y = linear(r[0] if save else r, w_out, workspace=workspace, stream=stream)
    return (y, r[1]) if save else y


def feed_forward_backward(dy, x, w_in, w_out, pre, activation="silu", workspace=None, stream=None):
    """Gradients (dx, dw_in, dw_out) of feed_forward from dy (m, k); gated's output is
    formed again from pre."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return feed_forward_backward(dy, x, w_in, w_out, pre, activation, workspace)
    r = mx._native().feed_forward_backward(dy, x, w_in, w_out, pre, activation,
                                           _buffer(workspace, x))
    if r.__class__ is int:
        raise SkgError(r, "skg_feed_forward_backward")
    return r
