"""The oracle of the gated block and the 4-bit products: values that are known
without it, and gradients against differences."""
import math

import numpy as np
import pytest

from oracle import gated


@pytest.mark.parametrize("name", ["silu", "gelu", "relu", "none"])
def test_slope_is_the_activation_s(name):
    x = np.linspace(-6, 6, 97) + 0.01
    d = 1e-5
    diff = (gated.act(x + d, name) - gated.act(x - d, name)) / (2 * d)
    assert np.allclose(gated.slope(x, name), diff, atol=1e-8)


def test_activation_values():
    assert gated.act(np.array([math.log(3.0)]), "silu")[0] == pytest.approx(0.75 * math.log(3.0), rel=1e-15)
    assert gated.slope(np.array([0.0]), "silu")[0] == 0.5
    assert gated.slope(np.array([0.0]), "gelu")[0] == 0.5
    assert gated.slope(np.array([-1.0, 0.0, 2.0]), "relu").tolist() == [0, 0, 1]


@pytest.mark.parametrize("name", ["silu", "gelu", "none"])
def test_gradients_against_differences(name):
    rng = np.random.default_rng(3)
    T, H, I = 3, 5, 4
    x, gate, up, dh = (rng.standard_normal(s) for s in ((T, H), (I, H), (I, H), (T, I)))

    def loss(x, gate, up):
        return (dh * gated.forward(x, gate, up, name, False)[0][0]).sum()

    got = gated.backward(dh, x, gate, up, x @ gate.T, x @ up.T, name, False)
    d = 1e-6
    for key, v in (("dx", x), ("dgate", gate), ("dup", up)):
        for at in np.ndindex(v.shape):
            a, b = v.copy(), v.copy()
            a[at] += d
            b[at] -= d
            args = {"dx": (x, gate, up), "dgate": (x, gate, up), "dup": (x, gate, up)}[key]
            lo, hi = list(args), list(args)
            k = ("dx", "dgate", "dup").index(key)
            hi[k], lo[k] = a, b
            assert (loss(*hi) - loss(*lo)) / (2 * d) == pytest.approx(got[key][0][at], rel=1e-6, abs=1e-8)


def test_beta_adds_what_was_there():
    rng = np.random.default_rng(4)
    x, gate, up, dh = (rng.standard_normal(s) for s in ((3, 5), (4, 5), (4, 5), (3, 4)))
    old = rng.standard_normal((4, 5))
    plain = gated.backward(dh, x, gate, up, x @ gate.T, x @ up.T, "silu", False)
    more = gated.backward(dh, x, gate, up, x @ gate.T, x @ up.T, "silu", False, 0.5, old, 2 * old)
    assert np.allclose(more["dgate"][0] - plain["dgate"][0], 0.5 * old)
    assert np.allclose(more["dup"][0] - plain["dup"][0], old)


def test_int4_by_hand():
    codes = np.array([[0x21, 0x0F], [0x80, 0xF0]], np.uint8)      # rows 1 2 15 (0) and 0 8 0 (15)
    assert gated.unpack(codes, 3).tolist() == [[1, 2, 15], [0, 8, 0]]
    scales = np.array([[0.5, 2.0]])
    w, most = gated.int4_weights(codes, scales, None, 3, 32)
    assert w.tolist() == [[-3.5, -3.0, 3.5], [-16, 0, -16]]
    assert most.tolist() == [[4.5, 5, 11.5], [16, 32, 16]]
    w, _ = gated.int4_weights(codes, scales, np.array([[1, 15]]), 3, 32)
    assert w.tolist() == [[0, 0.5, 7.0], [-30, -14, -30]]
    y, _ = gated.int4_product(np.array([[1.0, 1, 1]]), w, most, False, 32)
    assert y.tolist() == [[7.5, -74]]
