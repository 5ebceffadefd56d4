"""Bounds and inputs shared by the tests of MX8 rows, the RMS norm and the matrix product.

A result of T is accepted within half a spacing of T around the oracle's value
plus ``delta``, as in ``_training.py``; u = 2**-24.  The deltas:

  * z (and y without an activation): the terms are exact products, their sum is
    taken 16 terms (8-bit: 32) at a time: each step adds a group to the running sum and
    rounds or truncates what it aligns, so it is off by at most 2 u of the
    magnitudes so far (all of them together, at most ``z_scale``): 2 u (K / 16
    + 16) z_scale, the 16 for the cut of K (eight partial sums) and the bias.
  * an activation carries that on with its largest slope, below 1.2, and adds its
    own arithmetic: t is off by four roundings, 4 u |t|, which reaches y = z s(t)
    relatively (weight below 1); 2^x, the sum, 1/x and the product a few ulp, 16 u:
    (4 |t| + 16) u |y|; gelu: 1 + erf is off by 4 u absolutely: 4 u |z| (+ 16 u |y|)
    (Abramowitz and Stegun's 7.1.26 is off by 1.5e-7 = 2.5 u in erf, halved in z (1 + erf) / 2: 1.3 u |z| of it).
    Where s has run down to 0, y is taken as 0: 2**-100 covers it (and subnormals).
  * a slope: below 1.2 and made of at most three terms of that size, each off by
    (4 |t| + 16) u with |t| < 80 where it counts (s (1 - s) |t| < 0.25): 64 u.
    quick_gelu's and the tanh form's t' z s (1 - s) is below 1 as well.
  * dz is rounded to T in front of the products: half(T) |dz| each, so
    half(T) times the sum of the terms' magnitudes, and 64 u of it for the slope.
    dbias sums dz unrounded: 64 u for the slope and 128 u for the sum (float32, depth below 100).
  * MX8 of a float32 value that is within delta of the oracle's: the scale is that
    of a maximum within delta; half a spacing of E4M3 under the kernel's scale, plus delta.
"""
import numpy as np
import torch

from oracle import products as op
from tests._helpers import U32, _report, to_np64
from tests._training import DT, assert_within  # noqa: F401

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY100 = 2.0 ** -100


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def scale_bytes(s):
    return s.view(torch.uint8).cpu().numpy().astype(np.int64)


def mx8_f64(q, s):
    """What MX8 rows of any leading dimensions stand for, (rows, n)."""
    n = q.shape[-1]
    return op.mx8_values(q.float().double().cpu().numpy().reshape(-1, n), scale_bytes(s).reshape(-1, s.shape[-1]))


def assert_mx8(q, s, want, delta, what):
    """MX8 rows of float32 values within ``delta`` of ``want``."""
    want = want.reshape(-1, want.shape[-1])
    delta = np.broadcast_to(np.asarray(delta, dtype=np.float64), want.shape)
    b = scale_bytes(s).reshape(-1, s.shape[-1])
    lo = op.mx8_bytes(op.mx8_group_max(np.maximum(np.abs(want) - delta, 0)))
    hi = op.mx8_bytes(op.mx8_group_max(np.abs(want) + delta))
    assert ((b >= lo) & (b <= hi)).all(), f"{what}: scales"
    got = mx8_f64(q, s)
    k = 2.0 ** (127.0 - np.repeat(b, 32, axis=1)[:, : want.shape[1]])
    top = (np.abs(want) + delta) * k
    with np.errstate(divide="ignore"):
        half = 2.0 ** (np.maximum(np.floor(np.log2(np.where(top > 0, top, 1.0))), -6) - 4) / k
    tol = half + delta
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), _report(bad, got, want, tol, what)


def z_delta(k, scale):
    return 2 * U32 * (k / 16 + 16) * scale


def y_delta(z, y0, zd, act, alpha):
    """delta of act(z) for a z within zd; y0 = act(z)."""
    if act in ("none", "relu"):
        return zd
    d = 1.2 * max(1.0, abs(alpha) / 1.702 if act == "quick_gelu" else 1.0) * zd + TINY100
    if act == "gelu":
        return d + U32 * (4 * np.abs(z) + 16 * np.abs(y0))
    with np.errstate(invalid="ignore"):
        t = np.abs(op._inner(z, act, alpha)[0])
        return d + np.where(np.abs(y0) < 1e-30, 0.0, (4 * t + 16) * U32 * np.abs(y0))


def product_inputs(m, n, k, dtype, seed, bias=True, residual=True):
    g = torch.Generator().manual_seed(seed)
    t = DT[dtype]
    a = torch.randn(m, k, generator=g).to(t)
    w = (torch.randn(n, k, generator=g) / max(1, k) ** 0.5).to(t)
    b = torch.randn(n, generator=g).mul(0.3).to(t)
    r = torch.randn(m, n, generator=g).to(t)
    return a, w, b if bias else None, r if residual else None


def cuda(*tensors):
    out = tuple(None if t is None else t.cuda() for t in tensors)
    return out if len(out) > 1 else out[0]


def at_offset(t, elements):
    """A copy of t that starts ``elements`` elements off a 16-byte boundary."""
    if t is None:
        return None
    buf = torch.empty(t.numel() + elements, dtype=t.dtype, device=t.device)
    out = buf[elements:].view(t.shape)
    out.copy_(t)
    return out
