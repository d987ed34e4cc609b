"""CPU oracle of the 8-bit block-scaled matrices and the mixture-of-experts
layer, in binary64.

TEST INFRASTRUCTURE (see the package docstring). Definitions followed:

  e4m3   1 sign, 4 exponent, 3 mantissa bits, bias 7, largest value 448, no
         infinities, magnitude code 0x7F is NaN;
  quantise  s = max(fl32(max|x| / 448), 2^-126) over the block's finite
         elements; code = the e4m3 value nearest to x / s, ties to the even
         code; NaN and infinities give NaN;
  product   C = alpha * sum_b SA[b,i] SB[b,j] sum_{k in b} A[i,k] B[j,k]
         + beta C;
  layer  out_t = sum_s w[t,s] down_e (act(gate_e x_t) * (up_e x_t)).

A binary64 quotient of two binary32 values is within 2^-53 of the exact one,
and an exact quotient that is not the middle of two codes differs from it by
more than 2^-30 relative (x - s * middle is a multiple of both operands' last
bits), so deciding on the binary64 quotient decides on the exact one.

Bounds. A sum of n exact products in binary32, in any order and with any
rounding whose steps are at most one unit in the last place (2^-23 relative),
is off by at most n * 2^-23 * sum|products| to first order; every bound below
adds such terms with n the number of additions that a product passes.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
U = 2.0 ** -23      # one unit in the last place of binary32, relative
MAGNITUDES = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                       for e in range(16) for m in range(8)][:127])


def values(codes):
    """binary64 values of uint8 codes."""
    c = np.asarray(codes, dtype=np.uint8)
    mag = np.concatenate([MAGNITUDES, [np.nan]])[c & 0x7F]
    return np.where(c & 0x80, -mag, mag)


def nearest_codes(q):
    """uint8 codes of the e4m3 values nearest to binary64 q (|q| below 464),
    ties to the even code; NaN and infinities: 0x7F."""
    a = np.abs(q)
    bad = ~np.isfinite(a)
    a = np.where(bad, 0.0, a)
    mid = (MAGNITUDES[1:] + MAGNITUDES[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")     # first middle >= a: ties on the lower code
    at = np.minimum(lo, 125)
    lo = np.where((lo < 126) & (mid[at] == a) & (lo % 2 == 1), lo + 1, lo)
    code = lo.astype(np.uint8) | np.where(np.signbit(q), 0x80, 0).astype(np.uint8)
    return np.where(bad, 0x7F, code).astype(np.uint8)


def cdiv(a, b):
    return -(-a // b)


def quantize(x, tall):
    """(codes R x C, scales [column block, row or row block]) of binary32 x in
    tall x 128 blocks."""
    x = np.asarray(x, dtype=np.float32)
    R, C = x.shape
    codes = np.zeros((R, C), np.uint8)
    scales = np.zeros((cdiv(C, BLOCK), cdiv(R, tall)), np.float32)
    for i in range(cdiv(R, tall)):
        for b in range(cdiv(C, BLOCK)):
            blk = x[i * tall:(i + 1) * tall, b * BLOCK:(b + 1) * BLOCK].astype(np.float64)
            fin = np.abs(blk[np.isfinite(blk)])
            m = fin.max() if fin.size else 0.0
            s = max(np.float32(m / 448.0), np.float32(2.0 ** -126))
            scales[b, i] = s
            codes[i * tall:(i + 1) * tall, b * BLOCK:(b + 1) * BLOCK] = nearest_codes(
                blk / np.float64(s))
    return codes, scales


def stands_for(codes, scales, tall):
    """binary64 values of codes with scales [column block, row block]."""
    R, C = codes.shape
    s = scales.astype(np.float64)[np.arange(C)[None, :] // BLOCK, np.arange(R)[:, None] // tall]
    return values(codes) * s


def product(A, SA, B, SB, tallb, alpha=1.0, beta=0.0, C=None, narrow=False):
    """(C, bound of its binary32 error) in binary64. narrow: a block's sum may
    lose, of each product, what lies 2^-14 below the block's largest one."""
    a, b = stands_for(A, SA, 1), stands_for(B, SB, tallb)
    c = alpha * (a @ b.T)
    K = A.shape[1]
    # a product passes at most 128 additions in its block, the scaling (two
    # roundings), one addition per block and split, alpha and the beta term
    n = min(K, BLOCK) + 2 * cdiv(K, BLOCK) + 6
    bound = n * U * abs(alpha) * (np.abs(a) @ np.abs(b).T)
    if narrow:
        for k in range(0, K, BLOCK):
            most = np.abs(a[:, k:k + BLOCK]).max(1)[:, None] * np.abs(b[:, k:k + BLOCK]).max(1)
            bound = bound + abs(alpha) * min(K - k, BLOCK) * 2.0 ** -14 * most
    if beta != 0:
        c = c + beta * C
        bound = bound + 2 * U * np.abs(beta * C)
    return c, bound


def bf16_half_step(c):
    """Largest rounding error of bfloat16 results near c."""
    return np.abs(c) * 2.0 ** -8 + 2.0 ** -134


def act(x, name):
    import math
    if name == "silu":
        return x / (1 + np.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1 + np.vectorize(math.erf)(x / math.sqrt(2)))
    if name == "relu":
        return np.maximum(x, 0)
    return x


def top_k(logits, k):
    """ids by descending logit, ties to the lowest expert, NaN as -inf."""
    key = np.where(np.isnan(logits), -np.inf, logits)
    return np.argsort(-key, axis=1, kind="stable")[:, :k]


def route(x, router, k, renormalize):
    logits = x.astype(np.float64) @ router.astype(np.float64).T
    ids = top_k(logits, k)
    best = np.take_along_axis(logits, ids, 1)
    top = best[:, :1]
    over = best if renormalize else logits
    w = np.exp(best - top) / np.exp(over - top).sum(1, keepdims=True)
    return ids, w


def layer(x, gate, up, down, ids, w, activation="silu", h_bits=24):
    """(out, bound) for binary64 x [T, H], gate / up [E, I, H], down [E, H, I].
    h_bits: bits that the product with `down` keeps of h."""
    T, H = x.shape
    E, I = gate.shape[:2]
    out = np.zeros((T, H))
    bound = np.zeros((T, H))
    n1, n2 = H + 2 * cdiv(H, BLOCK) + 16, I + 2 * cdiv(I, BLOCK) + 16
    for t in range(T):
        for s in range(ids.shape[1]):
            e = int(ids[t, s])
            if e < 0 or e >= E:
                continue
            g, u = gate[e] @ x[t], up[e] @ x[t]
            # x and the weights are exact; a three-term split keeps 24 bits
            eg = n1 * U * (np.abs(gate[e]) @ np.abs(x[t]))
            eu = n1 * U * (np.abs(up[e]) @ np.abs(x[t]))
            a = act(g, activation)
            h = a * u
            # slopes of the activations are at most 1.13; the activation itself
            # is accurate to a few units in the last place, of 1 at worst
            eh = (1.13 * eg + 8 * U * np.maximum(np.abs(a), np.abs(g))) * np.abs(u) \
                + np.abs(a) * eu + eg * eu + (4 * U + 2.0 ** (1 - h_bits)) * np.abs(h)
            y = down[e] @ h
            ey = np.abs(down[e]) @ eh + n2 * U * (np.abs(down[e]) @ np.abs(h))
            out[t] += w[t, s] * y
            bound[t] += np.abs(w[t, s]) * (ey + (ids.shape[1] + 16) * U * np.abs(y))
    return out, bound
