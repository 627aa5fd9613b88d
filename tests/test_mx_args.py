"""Refusals of the microscaled entry points: argument errors come back
synchronously, before anything reaches a device (no GPU needed)."""
import pytest
import torch

from stream_decomposition_abft_gb300 import _build, mx, skgemm

P = 4096  # a plausible aligned address; never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return skgemm.lib()


def test_sizes():
    assert [skgemm.mx_codes_ld(k, skgemm.MXFP8) for k in (0, 1, 32, 33)] == [0, 32, 32, 64]
    assert [skgemm.mx_codes_ld(k, skgemm.NVFP4) for k in (0, 1, 32, 33)] == [0, 16, 16, 32]
    # Tiles of 128 rows x 4 blocks, 512 bytes each.
    assert skgemm.mx_scales_size(1, 1, skgemm.MXFP8) == 512
    assert skgemm.mx_scales_size(129, 128, skgemm.MXFP4) == 1024
    assert skgemm.mx_scales_size(128, 129, skgemm.MXFP8) == 1024
    assert skgemm.mx_scales_size(128, 128, skgemm.NVFP4) == 1024
    assert skgemm.mx_scales_size(0, 128, skgemm.NVFP4) == 0
    assert skgemm.mx_scales_size(-1, 1, 0) == 0 and skgemm.mx_codes_ld(-1, 0) == 0
    assert skgemm.mx_scales_size(1, 1, 3) == 0 and skgemm.mx_codes_ld(1, 3) == 0
    assert skgemm.workspace_size_mx(1, 1, 1, 3) == 0
    assert skgemm.workspace_size_mx(1, 1, 1, 0) == skgemm.workspace_size_mx(9999, 1, 777, 2) > 0


def test_quantize_arguments():
    def call(rows=4, k=64, X=P, ldx=None, dtype=skgemm.OUT_BF16, tr=0, fmt=0, g=None, codes=P,
             ldq=64, scales=P, values=None, ldv=0):
        ldx = (rows if tr else k) if ldx is None else ldx
        return skgemm.mx_quantize(rows, k, X, ldx, dtype, tr, fmt, g, codes, ldq, scales, values,
                                  ldv, None)
    assert call(rows=-1) == call(k=-1) == skgemm.ERR_ARG
    assert call(dtype=3) == call(dtype=-1) == call(fmt=3) == call(fmt=-1) == call(tr=2) == \
        skgemm.ERR_ARG
    assert call(rows=0) == call(k=0) == skgemm.OK
    assert call(X=None) == call(codes=None) == call(scales=None) == skgemm.ERR_ARG
    assert call(ldx=63) == call(ldq=48) == call(tr=1, rows=65, ldx=64) == skgemm.ERR_ARG
    assert call(values=P, ldv=63) == skgemm.ERR_ARG
    assert call(codes=P + 8) == call(scales=P + 8) == call(ldq=72) == skgemm.ERR_UNSUPPORTED
    assert call(X=P + 1) == call(g=P + 2, fmt=2) == skgemm.ERR_UNSUPPORTED
    assert call(k=1 << 30, ldq=1 << 30, ldx=1 << 30) == skgemm.ERR_UNSUPPORTED


def test_quantize_both_arguments():
    def call(rows=4, cols=64, X=P, ldx=64, dtype=skgemm.OUT_BF16, fmt=0, g=None, codes=P, ldq=64,
             scales=P, ct=P, ldt=32, st=P):
        return skgemm.mx_quantize_both(rows, cols, X, ldx, dtype, fmt, g, codes, ldq, scales, ct,
                                       ldt, st, None)
    assert call(rows=-1) == call(cols=-1) == call(dtype=3) == call(fmt=3) == skgemm.ERR_ARG
    assert call(rows=0) == call(cols=0) == skgemm.OK
    for name in ("X", "codes", "scales", "ct", "st"):
        assert call(**{name: None}) == skgemm.ERR_ARG
    assert call(ldx=63) == call(ldq=48) == call(ldt=16) == skgemm.ERR_ARG
    assert call(ct=P + 8) == call(st=P + 4) == call(ldt=40) == call(X=P + 1) == \
        skgemm.ERR_UNSUPPORTED


def test_norm_arguments():
    def call(rows=4, cols=64, X=P, ldx=64, res=None, ldr=0, w=P, dtype=0, eps=1e-5, s=None, lds=0,
             rstd=None, fmt=0, g=None, codes=P, ldq=64, scales=P):
        return skgemm.rmsnorm_mx(rows, cols, X, ldx, res, ldr, w, dtype, eps, s, lds, rstd, fmt, g,
                                 codes, ldq, scales, None)
    assert call(rows=-1) == call(cols=-1) == call(dtype=2) == call(fmt=3) == skgemm.ERR_ARG
    assert call(eps=-1.0) == call(eps=float("nan")) == skgemm.ERR_ARG
    assert call(rows=0) == call(cols=0) == skgemm.OK
    assert call(X=None) == call(w=None) == call(codes=None) == call(scales=None) == skgemm.ERR_ARG
    assert call(ldx=63) == call(res=P, ldr=63) == call(s=P, lds=63) == call(ldq=48) == \
        skgemm.ERR_ARG
    assert call(X=P + 1) == call(w=P + 1) == call(codes=P + 4) == call(rstd=P + 2) == \
        skgemm.ERR_UNSUPPORTED

    def back(rows=4, cols=64, dy=P, lddy=64, h=P, ldh=64, w=P, rstd=P, dr=None, lddr=0, dtype=0,
             dx=P, lddx=64, dw=P, ws=None, nbytes=0):
        return skgemm.rmsnorm_backward(rows, cols, dy, lddy, h, ldh, w, rstd, dr, lddr, dtype, dx,
                                       lddx, dw, ws, nbytes, None)
    assert back(rows=-1) == back(cols=-1) == back(dtype=2) == back(dw=None) == skgemm.ERR_ARG
    assert back(cols=0) == skgemm.OK
    for name in ("dy", "h", "w", "rstd", "dx"):
        assert back(**{name: None}) == skgemm.ERR_ARG
    assert back(lddy=63) == back(ldh=63) == back(lddx=63) == back(dr=P, lddr=63) == skgemm.ERR_ARG
    assert back(dy=P + 1) == back(dx=P + 1) == back(dw=P + 2) == skgemm.ERR_UNSUPPORTED
    assert skgemm.workspace_size_rmsnorm_backward(-1, 4) == 0


def test_product_arguments():
    def call(m=4, n=8, k=64, A=P, lda=64, SA=P, B=P, ldb=64, SB=P, C=P, ldc=8, fmt=0, out=2, ga=None,
             ws=None, nbytes=0):
        return skgemm.gemm_mx(m, n, k, 1.0, A, lda, SA, ga, B, ldb, SB, None, 0.0, C, ldc, fmt, out,
                              ws, nbytes, None)
    assert call(m=-1) == call(n=-1) == call(k=-1) == call(fmt=3) == call(out=3) == skgemm.ERR_ARG
    assert call(m=0) == call(n=0) == skgemm.OK
    assert call(A=None) == call(B=None) == call(SA=None) == call(SB=None) == call(C=None) == \
        skgemm.ERR_ARG
    assert call(lda=48) == call(ldb=48) == call(ldc=7) == skgemm.ERR_ARG
    assert call(A=P + 8) == call(SB=P + 8) == call(lda=72) == call(C=P + 1) == call(ga=P + 2) == \
        skgemm.ERR_UNSUPPORTED
    assert call() == call(ws=P, nbytes=16) == call(ws=P + 16, nbytes=1 << 20) == \
        skgemm.ERR_WORKSPACE


def test_binding_refusals():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="unknown format"):
        mx.quantize(x, "fp8")
    with pytest.raises(ValueError, match="CUDA tensor"):
        mx.quantize(x, "mxfp8")
    with pytest.raises(ValueError, match="matrix"):
        mx.quantize(x[0], "mxfp8")
    with pytest.raises(ValueError, match="dtype"):
        mx.quantize(x.double(), "mxfp8")
    with pytest.raises(ValueError, match="dtype"):
        mx.rmsnorm(x, x[0], 1e-5)
    q = mx.Matrix("mxfp8", 4, 64, torch.zeros(4, 64, dtype=torch.uint8),
                  torch.zeros(512, dtype=torch.uint8))
    ws = type("W", (), {"buf": x})
    with pytest.raises(ValueError, match="codes or scales"):
        mx.matmul(q, q, workspace=ws)
    with pytest.raises(ValueError, match="tensor is wanted"):
        mx.quantize(None, "mxfp8")
    with pytest.raises(ValueError, match="Matrix is wanted"):
        mx.matmul((), q, workspace=ws)


def test_stall_arguments():
    assert skgemm.mx_test_stall(-1) == skgemm.ERR_ARG
    assert skgemm.mx_test_stall(0, 0) == skgemm.OK
