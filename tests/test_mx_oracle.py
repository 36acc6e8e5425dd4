"""The MX FP4 and head-rotation oracle against facts outside itself."""
from fractions import Fraction

import numpy as np

import oracle.mx as X


def test_codes_by_exact_rationals():
    # every border, both neighbours of it in float32, and a sweep, by fractions
    mids = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    v = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(9)),
                        np.linspace(0, 8, 257, dtype=np.float32)]).astype(np.float64)
    got = X._codes(v)
    assert got.tolist() == [X.round_code(Fraction(float(a))) for a in v]
    assert X._codes(-v).tolist() == [g + 8 for g in got]
    # ties by hand: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    assert X._codes(mids.astype(np.float64)).tolist() == [0, 2, 2, 4, 4, 6, 6]


def test_scales_by_hand():
    def scale(v):
        return int(X.quantize_rows(np.array([[v]]))[1][0, 0])
    # 2^(s - 127) puts the largest magnitude in [4, 8)
    assert [scale(v) for v in (4.0, 7.99, 8.0, 1.0, -1.0, 0.0)] == [127, 127, 128, 125, 125, 0]
    assert scale(2.0 ** -149) == 0 and scale(2.0 ** -126) == 0
    assert scale(2.0 ** -124) == 1 and scale(float(np.finfo(np.float32).max)) == 252
    assert scale(np.nan) == 255 and scale(-np.inf) == 255


def test_round_trip_layout_and_pads():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 37))
    c, s = X.quantize_rows(x)
    assert c.shape == (3, 32) and s.shape == (3, 2)
    assert not c[:, 16 + 3:].any() and not (c[:, 16 + 2] >> 4).any()     # codes past column 37
    y = X.dequantize_rows(c, s, 37)
    c2, s2 = X.quantize_rows(y)
    # a block whose largest value rounded up to the next power moves its scale, no value
    assert np.array_equal(X.dequantize_rows(c2, s2, 37), y)
    assert np.abs(y - x).max() <= np.abs(x).max() / 4 + 1e-12            # 7.99 becomes 6
    for m in range(3):
        for k in range(37):
            byte = int(c[m, k // 2])
            code = byte >> 4 if k % 2 else byte & 15
            want = (-1) ** (code >> 3) * X.GRID[code & 7] * 2.0 ** (int(s[m, k // 32]) - 127)
            assert y[m, k] == want


def test_products_by_loops():
    rng = np.random.default_rng(2)
    xq, sx = X.quantize_rows(rng.standard_normal((2, 40)))
    wq, sw = X.quantize_rows(rng.standard_normal((3, 40)))
    x, w = X.dequantize_rows(xq, sx), X.dequantize_rows(wq, sw)
    y, mag = X.linear_w4a4(xq, sx, wq, sw)
    for m in range(2):
        for n in range(3):
            t = [Fraction(x[m, k]) * Fraction(w[n, k]) for k in range(40)]
            assert abs(float(sum(t)) - y[m, n]) < 1e-12 and abs(float(sum(map(abs, t))) - mag[m, n]) < 1e-12


def test_rotation_keeps_norms_and_composes():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 1, 8))
    a = rng.standard_normal((2, 3))
    for halves in (True, False):
        y, mag = X.qk_norm_rope(x, None, np.cos(a), np.sin(a), 0.0, halves)
        assert np.allclose((y * y).sum(2), 8) and (mag >= np.abs(y) - 1e-15).all()
        assert np.array_equal(y[:, :, 6:], X.qk_norm_rope(x, None, np.ones((2, 3)), np.zeros((2, 3)), 0.0, halves)[0][:, :, 6:])
        # the angle of a complex number made of a pair grows by the angle
        p, q = (np.arange(3), np.arange(3) + 3) if halves else (2 * np.arange(3), 2 * np.arange(3) + 1)
        z0, z1 = x[:, 0, p] + 1j * x[:, 0, q], y[:, 0, p] + 1j * y[:, 0, q]
        assert np.allclose(z1 / np.abs(z1), z0 / np.abs(z0) * np.exp(1j * a))
