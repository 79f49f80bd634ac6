"""Pins of the fp64 MX and norm reference (oracle/mx.py): hand-worked values, properties and differences."""
import numpy as np
import pytest

from oracle import mx


def test_tables():
    assert mx.values(mx.E4M3)[-1] == 448 and mx.values(mx.E4M3)[1] == 2.0 ** -9 and mx.values(mx.E4M3)[8] == 2.0 ** -6
    assert len(mx.values(mx.E2M1)) == 8


@pytest.mark.parametrize("u,code", [(0.25, 0), (0.26, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5, 6),
                                    (5.01, 7), (100, 7)])
def test_e2m1_ties_go_to_the_even_code(u, code):
    assert mx.round_codes(np.array([u]), mx.E2M1)[0] == code


@pytest.mark.parametrize("amax,fmt,byte", [(6.0, mx.E2M1, 127), (7.99, mx.E2M1, 127), (8.0, mx.E2M1, 128),
                                           (448.0, mx.E4M3, 127), (1.0, mx.E4M3, 119), (0.0, mx.E2M1, 0),
                                           (2.0 ** -149, mx.E4M3, 0), (3.4e38, mx.E2M1, 252), (np.inf, mx.E4M3, 255)])
def test_scale_bytes(amax, fmt, byte):
    assert mx.scale_byte(np.array([amax]), fmt)[0] == byte


def test_worked_block():
    v = np.zeros((1, 32))
    v[0, :4] = [12.0, -5.0, 0.9, -0.2]  # largest 12: 2^3, scale 2^1
    code, byte = mx.quantize(v, mx.E2M1)
    assert byte[0, 0] == 128 and list(byte[0, 1:]) == [0, 0, 0]
    # over 2: 6, -2.5 (tie to 2), 0.45 -> 0.5, -0.1 -> -0
    assert list(code[0, :4]) == [7, 8 + 4, 1, 8]
    assert list(mx.dequantize(code, byte, 4, mx.E2M1)[0]) == [12.0, -4.0, 1.0, 0.0]


def test_nan_block_stays_apart():
    v = np.ones((2, 70))
    v[0, 33] = np.nan
    v[1, 3] = -np.inf
    code, byte = mx.quantize(v, mx.E4M3)
    d = mx.dequantize(code, byte, 70, mx.E4M3)
    assert np.isnan(d[0, 32:64]).all() and (d[0, :32] == 1).all() and (d[0, 64:] == 1).all()
    assert np.isnan(d[1, :32]).all() and (d[1, 32:] == 1).all()


@pytest.mark.parametrize("fmt", [mx.E2M1, mx.E4M3])
def test_layout_round_trip(fmt):
    rng = np.random.default_rng(5)
    v = rng.standard_normal((131, 300))
    code, byte = mx.quantize(v, fmt)
    assert (mx.unpack_codes(mx.pack_codes(code, fmt), 131, 300, fmt) == code).all()
    buf = mx.pack_scales(byte, 131, 300)
    assert (mx.unpack_scales(buf, 131, 300) == byte).all()
    assert len(np.unique(mx.scale_index(256, 256))) == 256 * 8 == mx.scale_bytes(256, 256)
    # row 40, block 5: tile 1 of the first row of tiles, lane 8, group 1, place 1
    assert mx.scale_index(131, 300)[40, 5] == 512 + 16 * 8 + 4 + 1


def test_gradients_against_differences():
    rng = np.random.default_rng(6)
    h, w, dy, dh = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    dx, dw = mx.rmsnorm_grads(dy, h, w, 1e-3, dh)
    step = 1e-6  # central differences: error about step^2
    for i in range(3):
        for j in range(7):
            e = np.zeros_like(h)
            e[i, j] = step
            num = (dy * (mx.rmsnorm(h + e, w, 1e-3) - mx.rmsnorm(h - e, w, 1e-3))).sum() / (2 * step) + dh[i, j]
            assert abs(num - dx[i, j]) < 1e-8
    for j in range(7):
        e = np.zeros_like(w)
        e[j] = step
        assert abs((dy * (mx.rmsnorm(h, w + e, 1e-3) - mx.rmsnorm(h, w - e, 1e-3))).sum() / (2 * step) - dw[j]) < 1e-8
