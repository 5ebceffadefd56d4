"""Plain CPU oracle of GroupNorm and BiasDropout and of their gradients.

TEST INFRASTRUCTURE ONLY, as ``oracle/epilogue.py``: float64 NumPy from the
definitions in ``include/ep.h``, no code shared with the library.  (These two
ops of the contrib family have no manifest page.)  Beside each result come the
magnitudes that the tests' float32 error bounds are made of.
"""
from __future__ import annotations

import numpy as np

from .epilogue import _np

MULTIPLIER_0, MULTIPLIER_1 = 0xD2511F53, 0xCD9E8D57
WEYL_0, WEYL_1 = 0x9E3779B9, 0xBB67AE85


def _f64(a):
    return None if a is None else _np(a).astype(np.float64)


# ---------------------------------------------------------------------------
# GroupNorm, channels last
# ---------------------------------------------------------------------------

def _grouped(x, groups):
    """(N, positions..., C) -> (N, S, groups, D)."""
    n, c = x.shape[0], x.shape[-1]
    return x.reshape(n, -1, groups, c // groups)


def group_norm(X, gamma, beta, groups, epsilon, silu=False):
    """y, mean and 1/sqrt(var + eps) (each (N, groups)); population variance,
    eps = float64(float32(epsilon))."""
    x = _f64(X)
    g4 = _grouped(x, groups)
    mean = g4.mean(axis=(1, 3))
    d = g4 - mean[:, None, :, None]
    var = (d * d).mean(axis=(1, 3))
    with np.errstate(divide="ignore", invalid="ignore"):
        inv = 1.0 / np.sqrt(var + float(np.float32(epsilon)))
        u = (d * inv[:, None, :, None]).reshape(x.shape) * _f64(gamma)
        if beta is not None:
            u = u + _f64(beta)
        y = u / (1.0 + np.exp(-u)) if silu else u
    return dict(Y=y, mean=mean, inv_std_dev=inv, u=u)


def group_norm_grad(dY, X, gamma, beta, mean, inv_std_dev, groups, silu=False):
    """dX, dgamma, dbeta from the given statistics, and the magnitudes
    ``dX_scale``, ``dgamma_scale``, ``dbeta_scale``: the sums of the absolute
    values of the terms that each result is made of."""
    x, dy, g = _f64(X), _f64(dY), _f64(gamma)
    m = _f64(mean).reshape(x.shape[0], 1, groups, 1)
    r = _f64(inv_std_dev).reshape(x.shape[0], 1, groups, 1)
    h = ((_grouped(x, groups) - m) * r).reshape(x.shape)
    u = h * g + (0.0 if beta is None else _f64(beta))
    du = dy
    if silu:
        s = 1.0 / (1.0 + np.exp(-u))
        du = dy * s * (1.0 + u * (1.0 - s))
    axes = tuple(range(x.ndim - 1))
    dbeta, dgamma = du.sum(axis=axes), (du * h).sum(axis=axes)
    t, h4 = _grouped(du * g, groups), _grouped(h, groups)
    m1 = t.mean(axis=(1, 3), keepdims=True)
    m2 = (t * h4).mean(axis=(1, 3), keepdims=True)
    dx = (r * (t - m1 - h4 * m2)).reshape(x.shape)
    # |du|'s bound: sigmoid' of the activation is at most (1 + |u|)
    adu = np.abs(dy) * (1.0 + np.abs(u)) if silu else np.abs(dy)
    at = _grouped(adu * np.abs(g), groups)
    a1 = at.mean(axis=(1, 3), keepdims=True)
    a2 = (at * np.abs(h4)).mean(axis=(1, 3), keepdims=True)
    scale = (r * (at + a1 + np.abs(h4) * a2)).reshape(x.shape)
    return dict(dX=dx, dgamma=dgamma, dbeta=dbeta, dX_scale=scale,
                dgamma_scale=(adu * np.abs(h)).sum(axis=axes), dbeta_scale=adu.sum(axis=axes))


# ---------------------------------------------------------------------------
# BiasDropout
# ---------------------------------------------------------------------------

def philox4x32(counter, key, rounds=10):
    """The four output words for one counter (four words) and key (two words),
    in Python integers: each round multiplies words 0 and 2 by the round
    constants and mixes the halves of the products with words 1 and 3 and the
    key, which then moves on by its increments."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = MULTIPLIER_0 * c[0], MULTIPLIER_1 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + WEYL_0) & 0xFFFFFFFF, (k[1] + WEYL_1) & 0xFFFFFFFF]
    return c


def dropout_words(numel, seed, offset, first=0):
    """The 32-bit words of elements first..first+numel-1 (first a multiple of 4)."""
    lo, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    block = np.arange(first // 4, first // 4 + (numel + 3) // 4, dtype=np.uint64)
    c = [block & lo, block >> half, np.full_like(block, offset & 0xFFFFFFFF), np.full_like(block, offset >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c[0] * np.uint64(MULTIPLIER_0), c[2] * np.uint64(MULTIPLIER_1)
        c = [(b >> half) ^ c[1] ^ np.uint64(k0), b & lo, (a >> half) ^ c[3] ^ np.uint64(k1), a & lo]
        k0, k1 = (k0 + WEYL_0) & 0xFFFFFFFF, (k1 + WEYL_1) & 0xFFFFFFFF
    return np.stack(c, axis=1).reshape(-1)[:numel].astype(np.uint32)


def dropout_keep(numel, ratio, seed, offset, first=0):
    """keep(i) = word(i) < round((1 - ratio) 2^32), at least one word kept."""
    limit = max(1, round((1.0 - ratio) * 4294967296.0))
    return dropout_words(numel, seed, offset, first).astype(np.uint64) < np.uint64(limit)


def bias_dropout(X, ratio, seed, offset, bias=None, residual=None):
    """Y, the kept term alone (``kept``) and the mask (``keep``)."""
    x = _f64(X)
    keep = dropout_keep(x.size, ratio, seed, offset).reshape(x.shape)
    with np.errstate(invalid="ignore", over="ignore"):
        s = x if bias is None else x + _f64(bias)
        kept = np.where(keep, s / (1.0 - ratio), 0.0)
        y = kept if residual is None else kept + _f64(residual)
    return dict(Y=y, kept=kept, keep=keep)


def bias_dropout_grad(dY, ratio, seed, offset):
    """dX, dbias and dbias's sum of absolute values (``dbias_scale``)."""
    d = bias_dropout(dY, ratio, seed, offset)
    axes = tuple(range(d["Y"].ndim - 1))
    return dict(dX=d["Y"], keep=d["keep"], dbias=d["Y"].sum(axis=axes), dbias_scale=np.abs(d["Y"]).sum(axis=axes))
