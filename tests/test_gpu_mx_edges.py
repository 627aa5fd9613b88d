"""Ends of the microscaled operators' ranges and of their Python interface, on the GPU."""
import os
import re

import numpy as np
import pytest
import torch

from oracle import mx_ref as mr
from stream_decomposition_abft_gb300 import mx, skgemm

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def randn(*shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("cols", [264, 1111, 4096, 16384, 40000])
@pytest.mark.parametrize("eps,size", [(float("inf"), 1.0), (3.4028e38, 2.0 ** 56)])
def test_norm_statistics_that_overflow(cols, eps, size):
    # mean(h^2) + eps is infinite, though the sum of h^2 is not: 1 / sqrt of it is 0, and so
    # is the output.
    x = torch.full((3, cols), size, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    q, _, rstd = mx.rmsnorm(x, w, eps)
    if eps < float("inf"):
        assert float(x[0].float().square().sum()) < 3.4e38
    assert rstd.tolist() == [0.0] * 3
    assert not bool(q.codes.any()) and not bool(q.scales.any())


def test_norm_of_empty_rows():
    # The mean over no elements is NaN; rstd is written for every row.
    rstd = torch.full((5,), 7.0, device="cuda")
    x = torch.empty(5, 8, dtype=torch.bfloat16, device="cuda")
    p = x.data_ptr()
    st = skgemm.rmsnorm_mx(5, 0, p, 8, None, 0, p, skgemm.IN_BF16, 1e-5, None, 0, rstd.data_ptr(),
                           skgemm.MXFP8, None, p, 0, p, torch.cuda.current_stream().cuda_stream)
    assert st == skgemm.OK
    assert bool(torch.isnan(rstd).all())
    q, h, rstd = mx.rmsnorm(x[:, :0], x[0, :0], 1e-5, residual=x[:, :0])
    assert q.codes.shape == (5, 0) and h.shape == (5, 0)
    assert rstd.shape == (5,) and bool(torch.isnan(rstd).all())


def test_flags_without_a_truth_value():
    x = randn(4, 64, seed=1)
    two = torch.ones(2, dtype=torch.bool)
    with pytest.raises(ValueError, match="transpose"):
        mx.quantize(x, "mxfp8", transpose=two)
    with pytest.raises(ValueError, match="values"):
        mx.quantize(x, "mxfp8", values=two)


def test_report_of_calls_without_a_workspace():
    a, b = mx.quantize(randn(40, 512, seed=1), "mxfp8"), mx.quantize(randn(300, 512, seed=2), "mxfp8")
    ws = mx.default_workspace()
    assert mx.default_workspace(a.codes.device) is ws
    ws.report(reset=True)
    want = mx.matmul(a, b, workspace=mx.workspace())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [mx.matmul(a, b), mx.matmul(a, b, stream=s), mx.linear(randn(3, 512, seed=3), b)]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], want)
    rep = ws.report(reset=True)
    assert rep.launches == 3 and rep.timeouts == 0 and rep.status_bits == 0
    # Captured: the graph's launches are counted there as well.
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mx.matmul(a, b)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and ws.report().launches == 2


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("m,n,k", [(5, 9, 32), (5, 9, 72), (40, 200, 40), (140, 150, 352),
                                   (600, 600, 288)])
def test_product_reads_no_scales_past_the_end(fmt, m, n, k):
    # NaN in every scale byte that the storage rules leave open: rows past m and n, blocks
    # past k (mxfp8), or past the multiple of 64 elements that a 4-bit instruction spans.
    span = 32 if fmt == "mxfp8" else 64
    live = -(-k // span) * span // mr.BLOCK[fmt]
    nb = -(-k // 32) * 32 // mr.BLOCK[fmt]
    groups = -(-nb // 4)
    ops = []
    for rows, seed in ((m, 1), (n, 2)):
        x = randn(rows, k, seed=seed, dtype=torch.float32)
        codes, scales = mr.quantize(x.cpu().numpy(), fmt)
        stored = np.full(-(-rows // 128) * groups * 512, 0x7F if fmt == "nvfp4" else 0xFF, np.uint8)
        r, b = np.meshgrid(np.arange(rows), np.arange(min(live, groups * 4)), indexing="ij")
        stored[mr.scale_offset(r, b, groups)] = 0
        r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
        stored[mr.scale_offset(r, b, groups)] = scales
        q = mx.Matrix(fmt, rows, k, torch.from_numpy(mr.pack(codes, fmt)).cuda(),
                      torch.from_numpy(stored).cuda())
        zeros = torch.from_numpy(mr.tile_scales(scales)).cuda()
        ops.append((q, q._replace(scales=zeros)))
    got = mx.matmul(ops[0][0], ops[1][0], out_dtype=torch.float32)
    want = mx.matmul(ops[0][1], ops[1][1], out_dtype=torch.float32)
    assert bool(torch.isfinite(got).all()) and torch.equal(got, want)


def test_readme_example():
    # The README's norm and linear layer run as they stand there, with the layers' results.
    with open(os.path.join(ROOT, "README.md")) as f:
        code = re.search(r"```python\n(.*?mx\.rmsnorm.*?)```", f.read(), re.S).group(1)
    m, k, n = 96, 256, 160
    env = dict(x=randn(m, k, seed=1), r=randn(m, k, seed=2), dy=randn(m, n, seed=3),
               w=randn(n, k, seed=4), norm_weight=1 + 0.1 * randn(k, seed=5))
    exec(code, env)
    h = env["x"].double() + env["r"].double()
    u = h / (h.square().mean(1, keepdim=True) + 1e-5).sqrt() * env["norm_weight"].double()
    dy, w = env["dy"].double(), env["w"].double()
    for got, want in ((env["y"], u @ w.t()), (env["dn"], dy @ w), (env["dw"], dy.t() @ u)):
        # Codes of e4m3 are within 1/16 of the values, independently: two of them in a product.
        assert float((got.double() - want).norm() / want.norm()) < 2 / 16
    dx, dnorm = mr.rmsnorm_backward(*(env[t].double().cpu().numpy() for t in
                                      ("dn", "h", "norm_weight", "rstd")))
    for got, want in ((env["dx"], dx), (env["dnorm"], dnorm)):
        # Of the given dn: one rounding to bf16.
        got = got.double().cpu().numpy()
        assert np.linalg.norm(got - want) / np.linalg.norm(want) < 2.0 ** -8


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("m,n", [(2048, 2041), (2048, 2042), (2048, 2045), (2300, 1923), (2300, 1990),
                                 (40000, 3), (40000, 7), (40000, 9), (300, 2047), (5, 1003)])
def test_product_leaves_what_is_behind_its_columns(fmt, dtype, m, n):
    # Rows of out on 16-byte boundaries, as many columns as leave whole 16 bytes unfilled, on
    # either kernel: the same bits as in rows of their own, and nothing behind them.
    a, b = mx.quantize(randn(m, 512, seed=m), fmt), mx.quantize(randn(n, 512, seed=n), fmt)
    buf = torch.full((m + 1, n // 8 * 8 + 24), 7.0, dtype=dtype, device="cuda")
    mx.matmul(a, b, out=buf[:m, 8:8 + n])
    assert torch.equal(buf[:m, 8:8 + n], mx.matmul(a, b, out_dtype=dtype))
    assert bool((buf[:, :8] == 7).all() and (buf[:, 8 + n:] == 7).all() and (buf[m] == 7).all())
