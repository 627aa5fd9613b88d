"""Ends of the microscaled operators' ranges and of their Python interface, on the GPU."""
import pytest
import torch

from stream_decomposition_abft_gb300 import mx, skgemm

pytestmark = pytest.mark.gpu


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
