"""QuickGelu in the product's epilogue, and its slope, for alpha of either sign and 0, at infinities too."""
import os

import numpy as np
import pytest
import torch

from oracle import products as op
from tests._helpers import U32
from tests._products import TINY100, assert_within, f64, y_delta

VALUES = [0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, 3.0, -3.0, 12.0, -12.0, 60.0, -60.0, 3e4, -3e4, 1e30, -1e30, float("inf"),
          float("-inf"), float("nan")]


def at_infinity(alpha):
    """Values and slopes at -infinity and +infinity, as the header states the first."""
    nan, inf = float("nan"), float("inf")
    return ((0.0, inf), (0.0, 1.0)) if alpha > 0 else ((-inf, 0.0), (1.0, 0.0)) if alpha < 0 else ((nan, nan), (nan, nan))


@pytest.mark.gpu
@pytest.mark.parametrize("alpha", [1.702, 0.25, 0.0, -0.25, -1.702])
@pytest.mark.parametrize("m", [1, 1040])
def test_limits(lib, m, alpha):
    n = 2568 if m > 1 else 72
    z = torch.tensor(VALUES)[torch.arange(n) % len(VALUES)].to(torch.bfloat16)
    a, w = torch.zeros(m, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 64, dtype=torch.bfloat16, device="cuda")
    y = lib.ep_matmul_bias_act(a, w, z.cuda(), activation=lib.EP_ACT_QUICK_GELU, alpha=alpha)[0]
    x = f64(z)
    low, high = at_infinity(alpha)[0]
    with np.errstate(invalid="ignore"):
        want = np.where(x == -np.inf, low, np.where(x == np.inf, high, op.activation(x, "quick_gelu", alpha)))
    fin = np.nan_to_num(x, posinf=0, neginf=0)
    delta = y_delta(fin, np.nan_to_num(want, posinf=0, neginf=0), 0.0, "quick_gelu", alpha)
    assert_within(y, np.broadcast_to(want, (m, n)), np.broadcast_to(delta, (m, n)), "quick_gelu limits")
    if m > 1:
        return
    d = lib.ep_matmul_bias_act_grad(torch.ones(1, n, dtype=torch.bfloat16, device="cuda"), a, w, z.view(1, n).cuda(),
                                    lib.EP_ACT_QUICK_GELU, alpha, dA=None, dW=None, dbias=True)[2]
    low, high = at_infinity(alpha)[1]
    with np.errstate(invalid="ignore", over="ignore"):
        far = np.abs(alpha * fin) > 700  # s (1 - s) z is 0 there, and 0 times infinity to float64
        t = np.where(far, 0.0, alpha * fin)
        s = 1 / (1 + np.exp(-np.where(far, np.sign(alpha * fin) * 700, t)))
        slope = np.where(far, np.where(alpha * fin > 0, 1.0, 0.0), s + t * s * (1 - s))
    slope = np.where(np.isnan(x), np.nan, np.where(x == -np.inf, low, np.where(x == np.inf, high, slope)))
    assert_within(d, slope, 64 * U32 + TINY100, "quick_gelu slope limits")


def test_the_header_says_so():
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ep.h"), encoding="utf-8") as f:
        text = " ".join(f.read().replace(" * ", " ").split())
    assert "all are 0 at" not in text
    assert "EP_ACT_QUICK_GELU where alpha > 0: with alpha < 0 it is 0 at +infinity and -infinity at -infinity, with alpha = 0 NaN" in text
