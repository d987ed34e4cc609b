"""CPU oracle of the gated feed-forward block and of products with 4-bit weights,
in binary64.

TEST INFRASTRUCTURE (see the package docstring). Definitions followed:

  forward   G = x gate^T, U = x up^T, h = act(G) * U;
  backward  dU = dh * act(G), dG = dh * U * act'(G), dx = dG gate + dU up,
            dgate = dG^T x + beta dgate, dup = dU^T x + beta dup;
  int4      w(n,c) = s(c // group, n) * (q(n,c) - z(c // group, n)), out = x w^T.

Bounds. As in oracle/lowp.py: a sum of n products in binary32 is off by at most n
units in the last place (U = 2^-23, relative) of the sum of magnitudes, in any order;
n counts the additions that a product passes. Activations and their slopes come from
hardware exponentials and reciprocals of about one unit each; an exponential of v is
off by (|v| + 2) U relative (its argument is rounded once, relative), and gelu's
erf by 4e-7. Values that are rounded to a type are off by half a step of it.
"""
from __future__ import annotations

import math

import numpy as np

from .lowp import U, act, cdiv, quantize, stands_for  # noqa: F401

_erf = np.vectorize(math.erf, otypes=[float])


def half_step(v, bf16):
    """Largest error of rounding v to bfloat16 (else to binary32)."""
    return np.abs(v) * (2.0 ** -8 if bf16 else 2.0 ** -24) + (2.0 ** -134 if bf16 else 2.0 ** -150)


def slope(x, name):
    """Derivative of the activation (relu: 0 at 0)."""
    if name == "silu":
        s = 1 / (1 + np.exp(-x))
        return s + x * s * (1 - s)
    if name == "gelu":
        return 0.5 * (1 + _erf(x / math.sqrt(2))) + x * np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if name == "relu":
        return (x > 0).astype(float)
    return np.ones_like(x)


def products(x, w, extra=16):
    """(x w^T, bound of its binary32 error)."""
    n = x.shape[1] + extra
    return x @ w.T, n * U * (np.abs(x) @ np.abs(w).T)


def act_error(g, a, name):
    """Bound of the activation's own error at g, value a."""
    if name in ("none", "relu"):
        return np.zeros_like(g)
    return (np.abs(g) + 8) * U * np.maximum(np.abs(a), 0.25 * np.abs(g))


def forward(x, gate, up, name, bf16):
    """((h, bound), (G, bound), (U, bound)); bounds include rounding to the type."""
    (g, eg), (u, eu) = products(x, gate), products(x, up)
    a = act(g, name)
    h = a * u
    ea = 1.13 * eg + act_error(g, a, name)     # slopes are at most 1.13
    eh = ea * np.abs(u) + np.abs(a) * eu + ea * eu + 4 * U * np.abs(h)
    out = lambda v, e: (v, e + half_step(np.abs(v) + e, bf16))  # noqa: E731
    return out(h, eh), out(g, eg), out(u, eu)


def backward(dh, x, gate, up, g, u, name, bf16, beta=0.0, dgate=0.0, dup=0.0):
    """{name: (value, bound)} of dx, dgate, dup and h for g and u as they were kept."""
    a, d = act(g, name), slope(g, name)
    ea = act_error(g, a, name)
    ed = (2 * np.abs(g) + 16) * U if name in ("silu", "gelu") else 0.0
    du, dg, h = dh * a, dh * u * d, a * u
    one = lambda v, e: e + half_step(np.abs(v) + e, bf16)  # noqa: E731
    edu = one(du, np.abs(dh) * ea + 2 * U * np.abs(du))
    edg = one(dg, np.abs(dh * u) * ed + 4 * U * np.abs(dg))
    res = {"h": (h, one(h, ea * np.abs(u) + 2 * U * np.abs(h)))}
    T, I = g.shape
    dx = dg @ gate + du @ up
    e = edg @ np.abs(gate) + edu @ np.abs(up)
    e = e + (2 * I + 32) * U * ((np.abs(dg) + edg) @ np.abs(gate) + (np.abs(du) + edu) @ np.abs(up))
    res["dx"] = (dx, one(dx, e))
    for key, v, ev, old in (("dgate", dg, edg, dgate), ("dup", du, edu, dup)):
        w = v.T @ x + beta * old
        e = ev.T @ np.abs(x) + (T + 32) * U * ((np.abs(v) + ev).T @ np.abs(x)) \
            + 2 * U * np.abs(beta * old)
        res[key] = (w, one(w, e))
    return res


def unpack(codes, K):
    """q of uint8 codes [N, ceil(K / 2)]."""
    q = np.stack((codes & 15, codes >> 4), axis=2).reshape(codes.shape[0], -1)
    return q[:, :K].astype(np.float64)


def int4_weights(codes, scales, zeros, K, group):
    """(w, |s| (q + z)) of codes [N, ceil(K / 2)], scales and zeros [groups, N]."""
    c = np.arange(K) // group
    q, s = unpack(codes, K), scales.astype(np.float64)[c].T
    z = 8.0 if zeros is None else zeros.astype(np.float64)[c].T
    return s * (q - z), np.abs(s) * (q + z)


def int4_product(x, w, most, bf16, group, rounded=True):
    """(x w^T, bound): sums of q x and of x apart, so magnitudes are those of q + z (sums of
    (q - z) x are within it)."""
    n = x.shape[1] + 2 * cdiv(x.shape[1], group) + 24
    y, e = x @ w.T, n * U * (np.abs(x) @ most.T)
    return y, (e + half_step(np.abs(y) + e, bf16) if rounded else e)
