"""Refusals of the projections' entry points: argument errors come back synchronously, before
anything reaches a device (no GPU needed)."""
import ctypes

import pytest
import torch

from stream_decomposition_abft_gb300 import _build, layers, mx, skgemm

P = 4096  # a plausible aligned address; never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return skgemm.lib()


def test_sizes():
    assert skgemm.workspace_size_layers() == skgemm.workspace_size_mx(1, 1, 1, 0) > 0
    assert skgemm.scratch_size_linear(0, 16) == skgemm.scratch_size_linear(-1, 16) == 0
    assert skgemm.scratch_size_linear(4, 0) == skgemm.scratch_size_linear(4, 520) == 0
    # t in two parts of two bytes, rank padded to 16; a plan for 256 rows.
    assert skgemm.scratch_size_linear(256, 8) - skgemm.scratch_size_linear(128, 16) == 128 * 16 * 4
    assert skgemm.scratch_size_linear(257, 16) - skgemm.scratch_size_linear(256, 16) > 256 * 36
    assert skgemm.scratch_size_gated_backward(-1, 8) == 0
    # DPRE, up to 128 rows twice; and H.
    assert skgemm.scratch_size_gated_backward(129, 64) == 129 * 64 * 4
    assert skgemm.scratch_size_gated_backward(128, 64) == 128 * 64 * 8
    assert skgemm.scratch_size_feed_forward_backward(256, 64) == 256 * 64 * 6
    assert skgemm.scratch_size_feed_forward_backward(64, 64) == 64 * 64 * 12
    assert skgemm.scratch_size_feed_forward_backward(0, 64) == 0


def test_linear_arguments():
    def call(m=4, n=16, k=64, X=P, ldx=64, W=P, ldw=64, ad=None, Y=P, ldy=16, dtype=1, ws=P,
             nbytes=1 << 20, sc=P, scb=1 << 20):
        return skgemm.linear(m, n, k, X, ldx, W, ldw, ad, Y, ldy, dtype, ws, nbytes, sc, scb, None)
    assert call(m=-1) == call(n=-1) == call(k=-1) == call(dtype=2) == call(dtype=-1) == skgemm.ERR_ARG
    assert call(m=0) == call(n=0) == skgemm.OK
    assert call(X=None) == call(W=None) == call(Y=None) == skgemm.ERR_ARG
    assert call(ldx=63) == call(ldw=56) == call(ldy=15) == skgemm.ERR_ARG
    assert call(X=P + 8) == call(W=P + 2) == call(Y=P + 4) == skgemm.ERR_UNSUPPORTED
    assert call(ldx=68) == call(ldw=65) == call(ldy=17) == skgemm.ERR_UNSUPPORTED
    assert call(m=1 << 30) == call(k=1 << 30, ldx=1 << 30, ldw=1 << 30) == skgemm.ERR_UNSUPPORTED
    assert call(ws=None) == call(ws=P + 16) == call(nbytes=64) == skgemm.ERR_WORKSPACE

    def adapters(**kw):
        a = dict(down=P, ld_down=64, stride_down=512, up=P, ld_up=8, stride_up=128, index=P,
                 scale=None, count=2, rank=8)
        a.update(kw)
        return skgemm.AdaptersArg(**a)
    assert ctypes.sizeof(skgemm.AdaptersArg) == 72

    def bad(**kw):
        return call(ad=adapters(**kw))
    assert bad(count=-1) == bad(rank=-8) == bad(index=None) == bad(down=None) == bad(up=None) == \
        skgemm.ERR_ARG
    assert bad(ld_down=56) == bad(ld_up=0) == bad(stride_down=0) == bad(stride_up=-8) == \
        skgemm.ERR_ARG
    assert bad(rank=12, ld_up=16) == bad(rank=520, ld_up=520) == bad(down=P + 8) == \
        bad(up=P + 8) == bad(ld_down=68) == bad(ld_up=12) == bad(stride_down=516) == \
        bad(stride_up=132) == bad(index=P + 2) == bad(scale=P + 1) == skgemm.ERR_UNSUPPORTED
    assert call(ad=adapters(), sc=None) == call(ad=adapters(), scb=64) == \
        call(ad=adapters(), sc=P + 16) == skgemm.ERR_WORKSPACE
    assert call(m=0, ad=adapters(index=None)) == skgemm.OK


def test_gated_arguments():
    def call(m=4, f=16, k=64, X=P, ldx=64, W=P, ldw=64, act=0, H=P, ldh=16, pre=None, ldp=0,
             dtype=0, ws=P, nbytes=1 << 20):
        return skgemm.gated(m, f, k, X, ldx, W, ldw, act, H, ldh, pre, ldp, dtype, ws, nbytes, None)
    assert call(m=-1) == call(f=-8) == call(k=-1) == call(dtype=2) == call(act=4) == call(act=-1) == \
        skgemm.ERR_ARG
    assert call(m=0) == call(f=0) == skgemm.OK
    assert call(X=None) == call(W=None) == call(H=None) == skgemm.ERR_ARG
    assert call(ldx=56) == call(ldw=56) == call(ldh=8) == call(pre=P, ldp=24) == skgemm.ERR_ARG
    assert call(f=12, ldh=16) == call(X=P + 8) == call(ldw=68) == call(ldh=20) == \
        call(pre=P + 8, ldp=32) == call(pre=P, ldp=36) == skgemm.ERR_UNSUPPORTED
    assert call(ws=None) == call(nbytes=8) == skgemm.ERR_WORKSPACE


def test_gradient_arguments():
    def dh(m=4, f=16, k=64, dH=P, lddh=16, X=P, ldx=64, W=P, ldw=64, pre=P, ldp=32, act=0, dX=P,
           lddx=64, dW=P, lddw=64, dtype=0, ws=P, nbytes=1 << 20, sc=P, scb=1 << 20):
        return skgemm.gated_backward(m, f, k, dH, lddh, X, ldx, W, ldw, pre, ldp, act, dX, lddx, dW,
                                     lddw, dtype, ws, nbytes, sc, scb, None)

    def dy(m=4, f=16, k=64, dY=P, lddy=64, X=P, ldx=64, Wi=P, ldwi=64, Wo=P, ldwo=16, pre=P, ldp=32,
           act=0, dX=P, lddx=64, dWi=P, lddwi=64, dWo=P, lddwo=16, dtype=0, ws=P, nbytes=1 << 20,
           sc=P, scb=1 << 20):
        return skgemm.feed_forward_backward(m, f, k, dY, lddy, X, ldx, Wi, ldwi, Wo, ldwo, pre, ldp,
                                            act, dX, lddx, dWi, lddwi, dWo, lddwo, dtype, ws, nbytes,
                                            sc, scb, None)
    for call in (dh, dy):
        assert call(m=-1) == call(f=-8) == call(k=-1) == call(dtype=2) == call(act=4) == \
            skgemm.ERR_ARG
        assert call(k=0) == call(m=0, f=0) == skgemm.OK
        assert call(X=None) == call(pre=None) == call(dX=None) == call(ldp=24) == call(lddx=56) == \
            skgemm.ERR_ARG
        assert call(f=12) == call(X=P + 2) == call(ldp=36) == call(dX=P + 8) == call(lddx=68) == \
            skgemm.ERR_UNSUPPORTED
        assert call(ws=None) == call(sc=None) == call(scb=256) == call(sc=P + 64) == \
            skgemm.ERR_WORKSPACE
    assert dh(dH=None) == dh(W=None) == dh(dW=None) == dh(lddh=8) == dh(ldw=56) == dh(lddw=56) == \
        skgemm.ERR_ARG
    assert dh(lddh=20) == dh(dW=P + 4) == dh(W=P + 8) == skgemm.ERR_UNSUPPORTED
    for name in ("dY", "Wi", "Wo", "dWi", "dWo"):
        assert dy(**{name: None}) == skgemm.ERR_ARG
        assert dy(**{name: P + 8}) == skgemm.ERR_UNSUPPORTED
    assert dy(lddy=56) == dy(ldwi=56) == dy(ldwo=8) == dy(lddwi=56) == dy(lddwo=8) == skgemm.ERR_ARG
    assert dy(ldwo=20) == dy(lddwo=20) == dy(ldwi=68) == skgemm.ERR_UNSUPPORTED


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    ws = type("W", (), {"buf": x})
    with pytest.raises(ValueError, match="CUDA tensor"):
        layers.linear(x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        layers.linear(x, x, workspace=ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        layers.gated(None, x)
    with pytest.raises(ValueError, match="tensor is wanted"):
        layers.gated(None, x, workspace=ws)
    with pytest.raises(ValueError, match="dtype"):
        layers.gated(x.float(), x, workspace=ws)
    with pytest.raises(ValueError, match="matrix is wanted"):
        layers.gated_backward(x, x[0], x, x, workspace=ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        layers.feed_forward_backward(x, x, x, x, x, workspace=ws)
    with pytest.raises(ValueError, match="arguments are wanted"):
        mx._native().linear(x, x)


def test_stall_arguments():
    assert skgemm.layers_test_stall(-1) == skgemm.ERR_ARG
    assert skgemm.layers_test_stall(0, 0) == skgemm.OK
