"""Outputs that share memory with an input or another output are refused before anything
reaches a device (no GPU needed); columns of one buffer beside one another are not."""
import random

import pytest

from stream_decomposition_abft_gb300 import _build, skgemm

MB = 1 << 20
WS, SC = 200 * MB, 210 * MB  # addresses that are never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    skgemm.lib()


def refused(st):
    # Past the checks a call without a device ends with ERR_CUDA; no call here has a device's
    # memory, so none may go on with one.
    return st == skgemm.ERR_ARG


linear_args = dict(m=8, n=16, k=64, X=1 * MB, ldx=64, W=2 * MB, ldw=64, ad=None, Y=3 * MB, ldy=16,
                   dtype=1, ws=WS, nbytes=MB, sc=SC, scb=MB)


def linear(**kw):
    a = dict(linear_args, **kw)
    return skgemm.linear(a["m"], a["n"], a["k"], a["X"], a["ldx"], a["W"], a["ldw"], a["ad"], a["Y"],
                         a["ldy"], a["dtype"], a["ws"], a["nbytes"], a["sc"], a["scb"], None)


def test_linear():
    assert refused(linear(Y=linear_args["X"])) and refused(linear(Y=linear_args["W"]))
    # The last bytes of x, and of out.
    assert refused(linear(Y=MB + 8 * 64 * 2 - 16)) and refused(linear(Y=MB - 16, ldy=16, m=1))
    # Columns of a buffer with rows of 128, of which x takes 0 to 63.
    assert refused(linear(ldx=128, Y=MB + 56 * 2, ldy=128))
    assert refused(linear(ldx=128, Y=MB + 120 * 2, ldy=128))  # its row ends in x's next
    assert refused(linear(ldx=128, Y=MB + 16, n=1, ldy=24))


def adapters(**kw):
    a = dict(down=10 * MB, ld_down=64, stride_down=512, up=11 * MB, ld_up=8, stride_up=128,
             index=12 * MB, scale=13 * MB, count=20, rank=8)
    return skgemm.AdaptersArg(**dict(a, **kw))


def test_adapters():
    assert refused(linear(ad=adapters(), Y=10 * MB)) and refused(linear(ad=adapters(), Y=11 * MB))
    assert refused(linear(ad=adapters(), Y=10 * MB + 19 * 1024 + 1008))  # the last matrix's end
    assert refused(linear(ad=adapters(), Y=12 * MB)) and refused(linear(ad=adapters(), Y=12 * MB + 16))
    assert refused(linear(ad=adapters(), Y=13 * MB + 64))  # scale's last value
    # One adapter has no stride.
    assert refused(linear(ad=adapters(count=1, stride_down=0), Y=10 * MB + 1008))


def test_gated_and_gradients():
    def gated(**kw):
        a = dict(X=1 * MB, W=2 * MB, H=3 * MB, P=4 * MB)
        a.update(kw)
        return skgemm.gated(4, 16, 64, a["X"], 64, a["W"], 64, 0, a["H"], 16, a["P"], 32, 0, WS, MB,
                            None)

    def dh(**kw):
        a = {n: (i + 1) * MB for i, n in enumerate(("dH", "X", "W", "P", "dX", "dW"))}
        a.update(kw)
        return skgemm.gated_backward(4, 16, 64, a["dH"], 16, a["X"], 64, a["W"], 64, a["P"], 32, 0,
                                     a["dX"], 64, a["dW"], 64, 0, WS, MB, SC, MB, None)

    def dy(**kw):
        a = {n: (i + 1) * MB for i, n in enumerate(("dY", "X", "Wi", "Wo", "P", "dX", "dWi", "dWo"))}
        a.update(kw)
        return skgemm.feed_forward_backward(4, 16, 64, a["dY"], 64, a["X"], 64, a["Wi"], 64, a["Wo"],
                                            16, a["P"], 32, 0, a["dX"], 64, a["dWi"], 64, a["dWo"],
                                            16, 0, WS, MB, SC, MB, None)
    for call, ins, outs in ((gated, ("X", "W"), ("H", "P")),
                            (dh, ("dH", "X", "W", "P"), ("dX", "dW")),
                            (dy, ("dY", "X", "Wi", "Wo", "P"), ("dX", "dWi", "dWo"))):
        for o in outs:
            for other in ins + outs:
                if o != other:
                    assert refused(call(**{o: 20 * MB, other: 20 * MB})), (call, o, other)
                    assert refused(call(**{o: 20 * MB, other: 20 * MB + 16})), (call, o, other)


def test_against_every_byte():
    """Strided matrices at random places of a small buffer: refused where a byte is shared, and
    only there."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("calls past the checks would reach the device")
    rng = random.Random(5)
    seen = [0, 0]
    for _ in range(4000):
        m, n, k = rng.randint(1, 5), rng.randint(1, 24), rng.choice((8, 16, 24))
        pitch = rng.choice((24, 32, 40, 48))
        ldy, ldx = pitch, rng.choice((pitch, pitch, 24, 56))
        Y, X = (MB + 16 * rng.randint(0, 30) for _ in range(2))
        ins = {X + 2 * (i * ldx + c) for i in range(m) for c in range(k)}
        outs = {Y + 2 * (i * ldy + c) for i in range(m) for c in range(n)}
        shared = bool(ins & outs)
        seen[shared] += 1
        st = linear(m=m, n=n, k=k, X=X, ldx=ldx, W=2 * MB, ldw=24, Y=Y, ldy=ldy)
        assert st == (skgemm.ERR_ARG if shared else skgemm.ERR_CUDA), (m, n, k, X - MB, ldx, Y - MB, ldy)
    assert min(seen) > 500


def test_strides_beyond_any_memory():
    """Refused by their size, before they are multiplied."""
    big = 1 << 61
    for ld in (1 << 39, 1 << 45, big):
        assert linear(ldx=ld) == linear(ldw=ld) == linear(ldy=ld) == skgemm.ERR_UNSUPPORTED
        for name in ("ld_down", "ld_up", "stride_down", "stride_up"):
            assert linear(ad=adapters(**{name: ld})) == skgemm.ERR_UNSUPPORTED, name
    assert linear(m=1 << 28, ldx=1 << 30) == skgemm.ERR_UNSUPPORTED
    assert skgemm.gated(4, 16, 64, MB, big, 2 * MB, 64, 0, 3 * MB, 16, None, 0, 0, WS, MB, None) == \
        skgemm.ERR_UNSUPPORTED
    assert skgemm.gated(4, 1 << 27, 64, MB, 64, 2 * MB, 1 << 34, 0, 3 * MB, 1 << 27, None, 0, 0, WS, MB,
                        None) == skgemm.ERR_UNSUPPORTED  # 2^28 rows
    # One row has no stride.
    assert linear(m=1, ldx=big, Y=MB) == skgemm.ERR_ARG
