"""Plain CPU oracle of MX8 rows, the RMS norm and the matrix product, and of
their gradients.

TEST INFRASTRUCTURE ONLY, as ``oracle/epilogue.py``: float64 NumPy from the
definitions in ``include/ep.h``, no code shared with the library.  Beside each
result come the magnitudes that the tests' error bounds are made of.
"""
from __future__ import annotations

import math

import numpy as np

GROUP = 32
MOST = 448.0
ACTS = ("none", "silu", "relu", "quick_gelu", "gelu", "fast_gelu")

_erfc = np.vectorize(math.erfc, otypes=[np.float64])  # 1 + erf has no digits left of its own below z = -8


# ---------------------------------------------------------------------------
# MX8
# ---------------------------------------------------------------------------

def e4m3_round(x):
    """float64 -> the nearest E4M3 value, ties to even (no magnitude above 464: none occurs here)."""
    a = np.abs(x)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6)
    step = 2.0 ** (e - 3)
    return np.rint(x / step) * step


def mx8_bytes(amax):
    """The scale's byte for the largest magnitude of a group."""
    with np.errstate(divide="ignore", invalid="ignore"):
        f, e = np.frexp(np.where(np.isfinite(amax), amax, 1.0))  # amax = f 2^e, 1/2 <= f < 1; 448 = 7/8 2^9
    b = np.where(amax > 0, e - 9 + (f > 0.875), -200) + 127
    return np.where(np.isinf(amax), 255, np.maximum(b, 1)).astype(np.int64)


def mx8_group_max(x):
    """The largest magnitude of each group of each row (NaN left out)."""
    rows, n = x.shape
    g = -(-n // GROUP)
    p = np.zeros((rows, g * GROUP))
    p[:, :n] = np.where(np.isnan(x), 0.0, np.abs(x))
    return p.reshape(rows, g, GROUP).max(axis=2)


def mx8_quantize(x):
    """(q as values, bytes) of float64 rows."""
    b = mx8_bytes(mx8_group_max(x))
    s = np.repeat(b, GROUP, axis=1)[:, : x.shape[1]]
    with np.errstate(invalid="ignore"):
        q = e4m3_round(np.where(s == 255, np.nan, x * 2.0 ** (127.0 - s)))
    return q, b


def mx8_values(q, b):
    s = np.repeat(b, GROUP, axis=1)[:, : q.shape[1]]
    return np.where(s == 255, np.nan, q * 2.0 ** (s - 127.0))


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------

def rms_norm(x, skip, gamma, bias, epsilon):
    """s, inv (rows, 1), y, and ``terms``: the sum of the magnitudes of s's terms."""
    s, t = x.copy(), np.abs(x)
    for a in (skip, bias):
        if a is not None:
            s = s + a
            t = t + np.abs(a)
    inv = 1.0 / np.sqrt((s * s).mean(axis=1, keepdims=True) + float(np.float32(epsilon)))
    return dict(s=s, inv=inv, y=s * inv * gamma, terms=t)


def rms_norm_grad(dy, s, gamma, inv, dsum=None):
    h, u = s * inv, dy * gamma
    m = (u * h).mean(axis=1, keepdims=True)
    dx = inv * (u - h * m)
    scale = inv * (np.abs(u) + np.abs(h) * np.abs(u * h).mean(axis=1, keepdims=True))
    if dsum is not None:
        dx = dx + dsum
        scale = scale + np.abs(dsum)
    return dict(dX=dx, dX_scale=scale, dgamma=(dy * h).sum(axis=0), dgamma_scale=np.abs(dy * h).sum(axis=0),
                dbias=dx.sum(axis=0), dbias_scale=scale.sum(axis=0))


# ---------------------------------------------------------------------------
# matrix product
# ---------------------------------------------------------------------------

def _gate(t):
    """1 / (1 + e^-t) and its complement."""
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-t)), 1.0 / (1.0 + np.exp(t))


def _inner(z, act, alpha):
    """t(z) and t'(z) of the activations z s(t)."""
    if act == "silu":
        return z, np.ones_like(z)
    if act == "quick_gelu":
        a = float(np.float32(alpha))
        return a * z, np.full_like(z, a)
    c = 2.0 * math.sqrt(2.0 / math.pi)
    return c * (z + 0.044715 * z ** 3), c * (1.0 + 3 * 0.044715 * z * z)


def activation(z, act, alpha=1.702):
    if act == "none":
        return z
    if act == "relu":
        return np.where(z < 0, 0.0, z)
    low = np.isneginf(z) if act != "quick_gelu" else np.isneginf(alpha * z)
    with np.errstate(invalid="ignore"):
        if act == "gelu":
            y = 0.5 * z * _erfc(-z / math.sqrt(2.0))
        else:
            y = z * _gate(_inner(z, act, alpha)[0])[0]
    return np.where(low, 0.0, y)


def activation_slope(z, act, alpha=1.702):
    if act == "none":
        return np.ones_like(z)
    if act == "relu":
        return np.where(z > 0, 1.0, 0.0)
    if act == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    t, d = _inner(z, act, alpha)
    s, r = _gate(t)
    return s + z * d * s * r


def matmul(a, w, bias=None, residual=None, act="none", alpha=1.702):
    """z, y and ``z_scale``: the sum of the magnitudes of z's terms."""
    z, scale = a @ w.T, np.abs(a) @ np.abs(w).T
    if bias is not None:
        z, scale = z + bias, scale + np.abs(bias)
    y = activation(z, act, alpha)
    return dict(z=z, z_scale=scale, y=y if residual is None else y + residual)


def matmul_grad(dy, a, w, z=None, act="none", alpha=1.702):
    """dz, dA, dW, dbias and the sums of the magnitudes of the terms of the last three."""
    dz = dy if act == "none" else dy * activation_slope(z, act, alpha)
    m = np.abs(dz)
    return dict(dz=dz, dA=dz @ w, dA_scale=m @ np.abs(w), dW=dz.T @ a, dW_scale=m.T @ np.abs(a), dbias=dz.sum(axis=0),
                dbias_scale=m.sum(axis=0))
