"""Bounds and inputs shared by the GroupNorm and BiasDropout tests.

A result of T is accepted within half a spacing of T around the oracle's value
plus ``delta``, the float32 error before that rounding (float32 results: delta
plus their own rounding, 2**-24 relative).  The deltas, in units of
u = 2**-24, from the arithmetic that the definitions need:

  * GroupNorm Y: the LayerNorm criterion 1e-5 (inputs of unit spread: |h| < 8,
    |gamma| < 2; a dozen roundings of values of at most 16, u each), plus
    4 u |mu| r |gamma| where the mean is large: mu is held in float32 and is off
    by its own rounding and by that of its sum.
  * mean: 16 u (|mu| + sigma); 1/sqrt(var + eps): 64 u relative (a sum of
    squares in float32: every term is positive, so its relative error is at most
    u times the depth of the summation, which is below 100 here, halved by the
    square root, and a few roundings).
  * dX: 64 u times the sum of the magnitudes of its terms (``dX_scale``): the
    two group means are sums of depth below 50, du takes some ten roundings.
  * dgamma, dbeta, dbias: 64 u times the sum of their terms' magnitudes, for
    the same reason.
  * BiasDropout: x + b, the scale 1 / (1 - ratio), and its product: 3 u of the
    kept term; the sum with the residual u of the result.
"""
import numpy as np
import torch

from tests._helpers import TINY, U32, _record, _report, to_np64, ulp16, ulp_bf16

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_spacing(o, dtype):
    if dtype == torch.float32:
        return U32 * np.abs(o) + TINY
    return 0.5 * (ulp16(o) if dtype == torch.float16 else ulp_bf16(o))


def assert_within(gpu, o, delta, what):
    """gpu within half a spacing (of its own type) of o, plus delta; NaN where o is NaN, and the same infinities."""
    g = to_np64(gpu).reshape(o.shape)
    delta = np.broadcast_to(np.asarray(delta, dtype=np.float64), o.shape)
    same = (np.isnan(g) & np.isnan(o)) | (np.isinf(o) & (g == o))
    with np.errstate(invalid="ignore"):
        tol = half_spacing(np.abs(o) + delta, gpu.dtype) + delta
        bad = ~same & ~(np.abs(g - o) <= tol)
    assert not bad.any(), _report(bad, g, o, tol, what)
    return _record(what, gpu.dtype, g, o, tol, np.isfinite(o))


def norm_delta(mean, inv, gamma, groups, channels):
    """delta of Y per sample and channel, (N, 1, C)."""
    per = channels // groups
    big = np.abs(mean * inv).repeat(per, axis=1)[:, None, :]
    return 1e-5 + 4 * U32 * big * np.abs(to_np64(gamma))


def group_norm_inputs(shape, dtype, seed, beta=True, mean=0.0, std=1.0):
    """X ~ N(mean, std) with channels of their own offset, gamma ~ U(0.5, 1.5), beta ~ N(0, 0.1), dY ~ N(0, 1)."""
    g = torch.Generator().manual_seed(seed)
    c = shape[-1]
    x = torch.randn(shape, generator=g) * std + mean + 0.3 * torch.randn(c, generator=g) * std
    gamma = torch.rand(c, generator=g) + 0.5
    b = torch.randn(c, generator=g) * 0.1
    dy = torch.randn(shape, generator=g)
    t = DT[dtype]
    return dict(X=x.to(t), gamma=gamma.to(t), beta=b.to(t) if beta else None, dY=dy.to(t))


def dropout_inputs(shape, dtype, seed, bias=True, residual=True):
    g = torch.Generator().manual_seed(seed)
    t = DT[dtype]
    x = torch.randn(shape, generator=g).to(t)
    x[x == 0] = 1.0   # a kept element is never 0, so the mask can be read off the result
    b = torch.randn(shape[-1], generator=g).mul(0.1).to(t) if bias else None
    r = torch.randn(shape, generator=g).to(t) if residual else None
    return dict(X=x, bias=b, residual=r)
