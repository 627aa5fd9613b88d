"""The block-scaled product's bounded waits: copies that never come make them run out, the
launch ends by itself with the time-out in its report, and the device stays usable."""
import pytest
import torch

from stream_decomposition_abft_gb300 import mx, skgemm

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def unstalled():
    yield
    assert skgemm.mx_test_stall(0) == skgemm.OK


# (m, n, k, stages that a CTA loads; it would need more). A tile of a CTA's own, from
# registers and through shared memory; tiles shared by 8 and by 4 CTAs; CTA pairs of one
# tile each, and of several (the first one whole).
@pytest.mark.parametrize("m,n,k,stages", [(128, 8192, 512, 1), (40, 1001, 384, 1),
                                          (1, 1024, 8192, 1), (1, 1024, 16384, 7),
                                          (512, 512, 8192, 1), (333, 1000, 2200, 1),
                                          (2048, 2048, 2048, 1), (2048, 2048, 2048, 7),
                                          (6000, 6000, 1024, 9)])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
def test_wait_runs_out(fmt, m, n, k, stages):
    g = torch.Generator(device="cuda").manual_seed(m + k)
    a, b = (mx.quantize(torch.randn(r, k, generator=g, device="cuda"), fmt) for r in (m, n))
    ws = mx.workspace()
    want = mx.matmul(a, b, workspace=ws)
    rep = ws.report(reset=True)
    assert rep.status_bits == 0 and rep.launches == 1
    # Each wait is left a hundred times what any of these products takes.
    assert skgemm.mx_test_stall(stages, 10_000_000) == skgemm.OK
    mx.matmul(a, b, workspace=ws)
    rep = ws.report(reset=True)  # waits for the launch
    assert rep.status_bits == 1 << skgemm.ERR_PIPELINE_TIMEOUT
    assert rep.timeouts >= 1 and rep.launches == 1
    # The next call on the same workspace is whole again.
    assert skgemm.mx_test_stall(0) == skgemm.OK
    assert torch.equal(mx.matmul(a, b, workspace=ws), want)
    rep = ws.report()
    assert rep.status_bits == 0 and rep.timeouts == 0
