"""Gated feed-forward block and low-rank adapters in float64 (test
infrastructure, as the rest of this package): the formulas as they are written,
and bounds of what float32 sums and one rounding per output may differ by.
"""
from __future__ import annotations

import math

import numpy as np

F32 = 2.0 ** -24                                    # half a step of float32
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # relative, of one rounding
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}     # half a step of the subnormals
_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(g, name):
    """act(g) and act'(g)."""
    g = np.asarray(g, dtype=np.float64)
    if name == "silu":
        s = np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))
        return g * s, s + g * s * (1 - s)
    if name == "gelu":
        phi = 0.5 * (1 + _erf(g / math.sqrt(2)))
        return g * phi, phi + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = np.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def forward(x, w, name, delta=None):
    """h, [G | U] and a bound of each one's float32 error (before rounding)."""
    K = x.shape[1]
    gu, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    # a float32 sum of K products in any order is off by at most K half steps
    # of the sum of magnitudes (the products of 16-bit values are exact in it)
    err = (K + 2) * F32 * mag
    if delta is not None:
        gu, err = gu + delta, err + F32 * (np.abs(gu) + np.abs(delta))
    return gated(gu, err, name)


def gated(gu, err, name):
    I = gu.shape[1] // 2
    g, u = gu[:, :I], gu[:, I:]
    a, _ = act(g, name)
    # |act'| <= 1.13 for all three; the activation itself is evaluated in some
    # ten float32 operations, with absolute error below 16 half steps of |g|
    h = a * u
    eh = (1.13 * err[:, :I] + 16 * F32 * np.abs(g)) * (np.abs(u) + err[:, I:]) + np.abs(a) * err[:, I:] + 2 * F32 * np.abs(h)
    return h, gu, eh, err


def backward(dh, x, w, gu, name, dtype, tiny=None):
    """dx, dW, [dG | dU] and bounds of their errors before the last rounding.
    tiny: half a step of the smallest values of the rounded [dG | dU] that the
    products take (default: of the plain type)."""
    I = gu.shape[1] // 2
    g, u = gu[:, :I], gu[:, I:]
    a, da = act(g, name)
    d = np.concatenate([dh * u * da, dh * a], axis=1)
    # act' in some twenty float32 operations on values up to 1 + |g|, then one
    # rounding to the operands' type
    scale = np.concatenate([np.abs(dh * u) * (1 + np.abs(g)), np.abs(dh * g)], axis=1)
    ed = 32 * F32 * scale
    er = ed + HALF_STEP[dtype] * np.abs(d) + (TINY[dtype] if tiny is None else tiny)
    n, m = d.shape[1], d.shape[0]
    dx, dw = d @ w, d.T @ x
    ex = er @ np.abs(w) + (n + 2) * F32 * (np.abs(d) @ np.abs(w))
    ew = er.T @ np.abs(x) + (m + 2) * F32 * (np.abs(d).T @ np.abs(x))
    return (dx, dw, d), (ex, ew, ed)


def lora(x, a, b, ids, scaling, base, dtype):
    """out and a bound of its error before the last rounding."""
    M, N = x.shape[0], b.shape[1]
    K, R = a.shape[2], a.shape[1]
    out = np.zeros((M, N)) if base is None else np.array(base, dtype=np.float64)
    err = F32 * np.abs(out)
    for m in range(M):
        i = int(ids[m])
        if not 0 <= i < a.shape[0]:
            continue
        s = 1.0 if scaling is None else float(scaling[i])
        v = s * (a[i] @ x[m])
        # float32 sum over K and the scale, then two 16-bit terms: 2^-16 of the
        # value (bf16: 2^-8 of the 2^-8 that the first term leaves; f16: less)
        # and 2^-24 of the row's largest
        ev = abs(s) * (K + 4) * F32 * (np.abs(a[i]) @ np.abs(x[m])) + 2.0 ** -16 * np.abs(v) + 2.0 ** -24 * np.abs(v).max()
        out[m] += b[i] @ v
        err[m] += np.abs(b[i]) @ ev + (2 * R + 4) * F32 * (np.abs(b[i]) @ np.abs(v))
    return out, err + F32 * np.abs(out)


def within(got, want, err, dtype):
    """Elements of got (rounded once to dtype) outside err plus that rounding."""
    return ~(np.abs(got - want) <= err + HALF_STEP[dtype] * (np.abs(want) + err) + TINY[dtype])
