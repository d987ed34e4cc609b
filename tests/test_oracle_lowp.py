"""Pins of the 8-bit and mixture-of-experts oracle (oracle/lowp.py)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import lowp


def test_magnitudes_are_torch_e4m3():
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn).float()
    np.testing.assert_array_equal(lowp.values(np.arange(256)), t.numpy().astype(np.float64))
    assert lowp.MAGNITUDES[-1] == 448.0 and len(lowp.MAGNITUDES) == 127


def test_nearest_codes_of_codes_middles_and_neighbours():
    m = lowp.MAGNITUDES
    np.testing.assert_array_equal(lowp.nearest_codes(m), np.arange(127))
    np.testing.assert_array_equal(lowp.nearest_codes(-m), np.arange(127) | 0x80)
    mid = (m[1:] + m[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127))
    np.testing.assert_array_equal(lowp.nearest_codes(mid), even)
    np.testing.assert_array_equal(lowp.nearest_codes(np.nextafter(mid, 0)), np.arange(126))
    np.testing.assert_array_equal(lowp.nearest_codes(np.nextafter(mid, 999)), np.arange(1, 127))
    np.testing.assert_array_equal(lowp.nearest_codes(np.array([np.nan, np.inf, -np.inf])),
                                  [0x7F] * 3)


def test_quantize_against_exact_rationals():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 200)).astype(np.float32)
    x[1] *= 1e-30
    x[2, :] = 0
    codes, scales = lowp.quantize(x, 1)
    assert scales[0, 2] == np.float32(2.0 ** -126) and not codes[2].any()
    for i in range(5):
        for c in range(0, 200, 7):
            q = Fraction(float(x[i, c])) / Fraction(float(scales[c // 128, i]))
            d = [abs(abs(q) - Fraction(float(m))) for m in lowp.MAGNITUDES]
            assert d[int(codes[i, c]) & 0x7F] == min(d)


def test_product_and_layer_closed_forms():
    A = np.full((2, 130), lowp.nearest_codes(np.array([2.0]))[0], np.uint8)
    S = np.array([[1.0, 3.0], [0.5, 0.25]], np.float32)
    c, _ = lowp.product(A, S, A[:1], np.array([[2.0], [4.0]], np.float32), 128)
    # row 0: 128 * 4 * 1 * 2 + 2 * 4 * 0.5 * 4; row 1: 128 * 4 * 3 * 2 + 2 * 4 * 0.25 * 4
    np.testing.assert_array_equal(c, [[1040.0], [3080.0]])
    x = np.array([[1.0, 2.0]])
    gate = np.array([[[1.0, 1.0]], [[0.0, 1.0]]])
    up = np.array([[[1.0, 0.0]], [[2.0, 0.0]]])
    down = np.array([[[1.0], [2.0]], [[3.0], [-1.0]]])
    out, _ = lowp.layer(x, gate, up, down, np.array([[1, 0, -1]]), np.array([[0.5, 2.0, 9.0]]),
                        "relu")
    # expert 1: h = 2 * 2; expert 0: h = 3 * 1
    np.testing.assert_array_equal(out, [[0.5 * 12 + 2 * 3, 0.5 * -4 + 2 * 6]])
    assert lowp.top_k(np.array([[1.0, 5.0, 5.0, np.nan]]), 4).tolist() == [[1, 2, 0, 3]]
