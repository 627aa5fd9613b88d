"""C of n columns inside wider rows: what lies behind its columns stays as it was, whatever
number of them the last 16 bytes of a row hold."""
import pytest
import torch

from gpu_util import IN_CODE, OUT_CODE, check_full, reference, to_device
from stream_decomposition_abft_gb300 import inputs, skgemm

pytestmark = pytest.mark.gpu


def wide(p, opts, verify=False, status=0):
    """The call on C in rows of 16 bytes to 48 more than it needs; returns C."""
    per = 16 // torch.empty((), dtype=inputs.DTYPES[p.out_dtype]).element_size()
    ld = (p.n // per + 3) * per
    A, B = to_device(p, "cuda", p.A.shape[1] + -p.A.shape[1] % 8, p.B.shape[1] + -p.B.shape[1] % 8)
    buf = torch.full((p.m + 1, ld), 7.0, dtype=inputs.DTYPES[p.out_dtype], device="cuda")
    C = buf[:p.m, :p.n]
    if p.C0 is not None:
        C.copy_(p.C0.to("cuda"))
    ws = skgemm.Workspace(skgemm.workspace_size_layout(p.m, p.n, p.k, p.a_layout, p.b_layout, opts))
    fn = skgemm.gemm_verify if verify else skgemm.gemm
    st = fn(p.m, p.n, p.k, p.alpha, A.data_ptr(), A.stride(0), B.data_ptr(), B.stride(0), p.beta,
            C.data_ptr(), ld, IN_CODE[p.in_dtype], OUT_CODE[p.out_dtype], p.a_layout, p.b_layout,
            opts, ws.ptr, ws.nbytes, torch.cuda.current_stream().cuda_stream)
    assert st == skgemm.OK
    assert ws.report().status_bits == status
    assert bool((buf[:p.m, p.n:] == 7).all()) and bool((buf[p.m] == 7).all())
    return C


def problem(m, n, k, out, beta, **kw):
    return inputs.make_problem(m, n, k, seed=n, in_dtype="bf16", out_dtype=out, law_a="normal",
                               law_b="uniform", alpha=1.25, beta=beta, **kw)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("beta", [0.0, -0.5])
@pytest.mark.parametrize("m,n,k", [(200, 61, 136), (300, 1003, 520), (129, 257, 64), (1, 1, 8),
                                   (1000, 1301, 328), (77, 514, 1032), (5, 7, 8)])
def test_plans(out, beta, m, n, k):
    p = problem(m, n, k, out, beta)
    ref = reference(p)
    check_full(p, wide(p, None), ref)
    for tile_n, pair in ((64, 1), (128, 1), (256, 1), (256, 2)):
        for mode, g in (("dp", 4), ("sk", 6), ("sk2_dp", 8)):
            check_full(p, wide(p, skgemm.opts_default(sched=mode, tile_n=tile_n, cta_pair=pair,
                                                      grid=g)), ref)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("beta", [0.0, 0.75])
@pytest.mark.parametrize("extra", [dict(), dict(abft_local=2), dict(abft_inloop=2),
                                   dict(tile_n=256, cta_pair=2), dict(tile_n=256, cta_pair=1)])
@pytest.mark.parametrize("m,n,k", [(300, 1003, 520), (640, 765, 1536), (1024, 1021, 1024)])
def test_checked(out, beta, extra, m, n, k):
    p = problem(m, n, k, out, beta)
    check_full(p, wide(p, skgemm.opts_default(abft=1, **extra), verify=True))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("row,col", [(5, 1002), (3, 1000), (120, 999)])
def test_corrected_in_the_last_columns(out, row, col):
    # A fault in an element behind the last whole 16 bytes is found and put right there.
    p = problem(128, 1003, 512, out, 0.0)
    tiles_n = -(-1003 // 128)
    o = skgemm.opts_default(abft=1, tile_n=128, inject_tile=tiles_n - 1, inject_row=row,
                            inject_col=col - (tiles_n - 1) * 128, inject_bit=30)
    check_full(p, wide(p, o, status=1 << skgemm.ABFT_CORRECTED))


@pytest.mark.parametrize("layouts", [(1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("tile_n,pair", [(64, 1), (128, 1), (256, 1), (256, 2)])
def test_operands_along_either_dimension(layouts, tile_n, pair):
    p = problem(300, 1003, 520, "bf16", 0.5, a_layout=layouts[0], b_layout=layouts[1])
    check_full(p, wide(p, skgemm.opts_default(tile_n=tile_n, cta_pair=pair)))
