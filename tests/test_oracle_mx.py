"""Pins of the microscaled oracle to hand-computed values and to brute force."""
import numpy as np
import pytest

from oracle import mx_ref as mr


def test_tables():
    assert mr.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert len(mr.E4M3) == 127 and mr.E4M3[-1] == 448 and mr.E4M3[1] == 2.0 ** -9
    assert mr.E4M3[8] == 2.0 ** -6 and mr.E4M3[0x38] == 1.0


@pytest.mark.parametrize("y,want", [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6),
                                    (5.0, 6), (5.01, 7), (7.0, 7), (0.26, 1), (-2.6, 5)])
def test_e2m1_ties_to_even(y, want):
    assert int(mr.nearest_code(np.array([y]), mr.E2M1)[0]) == want


def test_nearest_is_nearest():
    rng = np.random.default_rng(0)
    y = rng.uniform(0, 448, 4000)
    got = mr.E4M3[mr.nearest_code(y, mr.E4M3)]
    assert np.array_equal(np.abs(got - y), np.abs(mr.E4M3[None] - y[:, None]).min(1))


@pytest.mark.parametrize("fmt,most", [("mxfp8", 448.0), ("mxfp4", 6.0)])
def test_power_of_two_scale(fmt, most):
    # The least 2^e with amax / 2^e <= most: exactly at most * 2^j it is 2^j, one
    # step above it 2^(j+1); zero blocks and subnormals get 2^-127 (byte 0).
    for j in (-3, 0, 5):
        for amax, e in ((most * 2.0 ** j, j), (np.nextafter(np.float32(most * 2.0 ** j),
                                                            np.float32(np.inf)), j + 1)):
            x = np.zeros((1, 32), dtype=np.float32)
            x[0, 7] = -amax
            codes, s = mr.quantize(x, fmt)
            assert int(s[0, 0]) == e + 127
            v = mr.values(codes, s, fmt, 1.0, 32)
            assert abs(v[0, 7] + amax) <= amax / 8
    assert int(mr.quantize(np.zeros((1, 32)), fmt)[1][0, 0]) == 0
    assert int(mr.quantize(np.full((1, 32), 1e-42, dtype=np.float32), fmt)[1][0, 0]) == 0


def test_nvfp4_scale_and_bad_blocks():
    x = np.zeros((2, 32), dtype=np.float32)
    x[0, 3], x[1, 20] = 12.0, np.nan
    codes, s = mr.quantize(x, "nvfp4", 0.5)
    # amax / (6 g) = 4 -> e4m3 code 0x48; 12 / (4 * 0.5) = 6 -> code 7.
    assert s.tolist() == [[0x48, 0], [0, 0x7F]] and int(codes[0, 3]) == 7
    v = mr.values(codes, s, "nvfp4", 0.5, 32)
    assert v[0, 3] == 12.0 and np.isnan(v[1, 16:]).all() and (v[1, :16] == 0).all()
    x[1, 20] = np.inf
    assert mr.quantize(x, "mxfp8")[1][1, 0] == 0xFF


def test_scale_tiles():
    # Row 32 q + l, block b of a tile at byte 16 l + 4 q + b.
    assert mr.scale_offset(0, 0, 3) == 0 and mr.scale_offset(1, 0, 3) == 16
    assert mr.scale_offset(32, 2, 3) == 6 and mr.scale_offset(127, 3, 3) == 511
    assert mr.scale_offset(0, 4, 3) == 512 and mr.scale_offset(128, 0, 3) == 3 * 512
    s = np.arange(1, 131 * 6 + 1).reshape(131, 6) % 251
    t = mr.tile_scales(s.astype(np.uint8))
    assert t.size == 2 * 2 * 512 and t[mr.scale_offset(130, 5, 2)] == s[130, 5]


def test_rmsnorm_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, r, w, dy = (rng.standard_normal(s) for s in ((3, 40), (3, 40), 40, (3, 40)))
    _, h, rstd = mr.rmsnorm(x, w, 1e-5, r)
    dx, dw = mr.rmsnorm_backward(dy, h, w, rstd)
    loss = lambda a, b: (mr.rmsnorm(a, b, 1e-5, r)[0] * dy).sum()
    for i, j in ((0, 0), (2, 17), (1, 39)):
        d = np.zeros_like(x)
        d[i, j] = 1e-6
        assert abs((loss(x + d, w) - loss(x - d, w)) / 2e-6 - dx[i, j]) < 1e-7
        e = np.zeros_like(w)
        e[j] = 1e-6
        assert abs((loss(x, w + e) - loss(x, w - e)) / 2e-6 - dw[j]) < 1e-7
