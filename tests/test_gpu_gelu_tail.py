"""The error-function GELU and its slope relative to their own size, at every float16 and bfloat16 z.

u = 2**-24.  With Phi(-|z|) = 1/2 e^(-z^2/2) t P(t), t = 1 / (1 + p |z|):
  * e^(-z^2/2): two products and a constant in its argument, 3 u z^2 / 2 (the argument's error is the result's
    relative error); 4 u for 2^x.
  * t: a constant, the sum, 2 u for 1/x: 4 u, which t P(t) takes up to 3.1 times (the derivative of its logarithm by
    log t is 3.03 at t = 1, its largest): 12.4 u; P's coefficients and sums, whose magnitudes add up to 1.6 of the
    value: 9 u; the fit 8.5 u.
  * the products by 1/2 t, e and z: 3 u.
  Altogether (37 + 1.5 z^2) u, 40 here; 1 - Phi(-|z|) is off by less, relatively.
  * the slope Phi + z phi: as much of the sum of its two terms' magnitudes, and the density's product, the sum and
    the product with dY: 44.
Below 2**-100 a result may be 0.
"""
import numpy as np
import pytest
import torch
from scipy.special import erfc

from tests._helpers import U32
from tests._products import DT, TINY100, assert_within, f64

pytestmark = pytest.mark.gpu


def every_value(dtype, most):
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(DT[dtype])
    v = v[v.isfinite() & (v.abs() <= most)]
    return v[: v.numel() // 8 * 8].cuda()


@pytest.mark.parametrize("m", [1, 260])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_value(lib, dtype, m):
    z = every_value(dtype, 14.0)
    a, w = torch.zeros(m, 8, dtype=z.dtype, device="cuda"), torch.zeros(z.numel(), 8, dtype=z.dtype, device="cuda")
    y = lib.ep_matmul_bias_act(a, w, z, activation=lib.EP_ACT_GELU)[0]
    assert torch.equal(y, y[:1].expand_as(y))
    x = f64(z)
    want = 0.5 * x * erfc(-x / np.sqrt(2.0))
    assert_within(y[0], want, (40 + 1.5 * x * x) * U32 * np.abs(want) + TINY100, "gelu tail")


@pytest.mark.parametrize("cut", [0, 3])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_slope(lib, dtype, cut):
    z = every_value(dtype, 14.0)
    z = z[: z.numel() - cut].view(1, -1).contiguous()
    n = z.numel()
    a, w = torch.zeros(1, 8, dtype=z.dtype, device="cuda"), torch.zeros(n, 8, dtype=z.dtype, device="cuda")
    d = lib.ep_matmul_bias_act_grad(torch.ones_like(z), a, w, z, lib.EP_ACT_GELU, dA=None, dW=None, dbias=True)[2]
    x = f64(z)[0]
    cdf, rest = 0.5 * erfc(-x / np.sqrt(2.0)), x * np.exp(-0.5 * x * x) / np.sqrt(2 * np.pi)
    assert_within(d, cdf + rest, (44 + 1.5 * x * x) * U32 * (cdf + np.abs(rest)) + TINY100, "gelu slope tail")
