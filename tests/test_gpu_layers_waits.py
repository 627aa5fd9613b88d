"""The bounded waits of a layer's projections: copies that never come make them run out, the
launches end by themselves with the time-out in the report, and the device stays usable."""
import pytest
import torch

from stream_decomposition_abft_gb300 import layers, skgemm

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def unstalled():
    yield
    assert skgemm.layers_test_stall(0) == skgemm.OK


def runs_out(call, launches, stages, ws):
    want = call()
    rep = ws.report(reset=True)
    launches = launches or rep.launches  # None: as many as the sizes have
    assert rep.status_bits == 0 and rep.launches == launches
    # Each wait is left a hundred times what any of these products takes.
    assert skgemm.layers_test_stall(stages, 10_000_000) == skgemm.OK
    call()
    rep = ws.report(reset=True)  # waits for the launches
    assert rep.status_bits == 1 << skgemm.ERR_PIPELINE_TIMEOUT
    assert rep.timeouts >= 1 and rep.launches == launches
    # The next call on the same workspace is whole again.
    assert skgemm.layers_test_stall(0) == skgemm.OK
    got = call()
    for a, b in zip(got if isinstance(got, tuple) else (got,),
                    want if isinstance(want, tuple) else (want,)):
        assert torch.equal(a, b)
    rep = ws.report()
    assert rep.status_bits == 0 and rep.timeouts == 0


def make(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


# Few rows, tiles shared by clusters, tiles of a CTA's own, CTA pairs of one and several tiles.
@pytest.mark.parametrize("m,n,k,stages", [(1, 1024, 8192, 1), (1, 1024, 8192, 7), (40, 1000, 2200, 1),
                                          (333, 1000, 2200, 2), (300, 8192, 512, 3),
                                          (2048, 2048, 2048, 1), (2048, 2048, 2048, 7),
                                          (6000, 6000, 1024, 17)])
def test_product(m, n, k, stages):
    ws, x, w = layers.workspace(), make(m, k), make(n, k, seed=1)
    runs_out(lambda: layers.linear(x, w, workspace=ws), 1, stages, ws)


# In one launch (few rows; more), in two (single CTAs, pairs); the down-projection's own wait.
@pytest.mark.parametrize("m,n,k,s,r,launches,stages", [
    (1, 1000, 8192, 4, 16, 1, 1), (8, 1000, 8192, 4, 16, 1, 5), (333, 1000, 2200, 5, 8, 1, 2),
    (64, 1000, 8192, 40, 16, 2, 1), (64, 1000, 8192, 40, 16, 2, 9), (300, 520, 1032, 40, 64, 2, 2),
    (2048, 4096, 1024, 40, 16, 2, 15), (16, 1000, 1032, 8, 200, 2, 2)])
def test_adapters(m, n, k, s, r, launches, stages):
    ws, x, w = layers.workspace(), make(m, k), make(n, k, seed=1)
    ad = layers.Adapters(make(s, r, k, seed=2), make(s, n, r, seed=3))
    i = (torch.arange(m, device="cuda") % s).int()
    runs_out(lambda: layers.linear(x, w, ad, i, workspace=ws), launches, stages, ws)


@pytest.mark.parametrize("m,f,k,stages", [(1, 1024, 8192, 2), (300, 520, 1032, 1), (2048, 2048, 1024, 9)])
def test_gated(m, f, k, stages):
    ws, x, w = layers.workspace(), make(m, k), make(2 * f, k, seed=1)
    runs_out(lambda: layers.gated(x, w, save=True, workspace=ws), 1, stages, ws)


@pytest.mark.parametrize("m,f,k,stages", [(100, 264, 520, 1), (323, 256, 520, 2), (300, 1800, 104, 4),
                                          (512, 2816, 1024, 3),
                                          (2048, 2048, 1024, 9)])
def test_gradients(m, f, k, stages):
    ws, x, wi, wo = layers.workspace(), make(m, k), make(2 * f, k, seed=1), make(k, f, seed=2)
    dy, pre = make(m, k, seed=3), make(m, 2 * f, seed=4)
    runs_out(lambda: layers.feed_forward_backward(dy, x, wi, wo, pre, workspace=ws), None,
             stages, ws)
