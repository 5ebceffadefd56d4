"""GroupNorm's SiLU and its derivative over the whole range of u.

With gamma = 0, u = beta exactly: y = silu(beta), and dbeta of one position with
dY = 1 is silu'(beta).  float32: 8 half steps of the result (sigmoid within 3 ulp, and
the products), and 2^-116 where the results near -87 have left the normal numbers'
reach of the sigmoid; 16 bits: half a spacing, and 16 half steps of float32 and |u|
2^-24 relatively for the hardware's 2^x and 1/x.  silu' = s (1 + u (1 - s)): 1 - s is
exact and takes over the error of s, which u multiplies; from u = 20 on s is 1 to
float32, and u (1 - s) < 5e-8.
"""
import numpy as np
import pytest
import torch

from tests._helpers import U32
from tests._training import DT, assert_within

pytestmark = pytest.mark.gpu

MOST = {"f32": 3.0e38, "f16": 65504.0, "bf16": 3.0e38}
# each in another form: few tokens, small samples (three ways), staged rows, staged odd rows, any C
SHAPES = [((1, 1, 2048), 8), ((1, 2, 2040), 8), ((1, 3, 2044), 28), ((1, 2, 2049), 3), ((1, 600, 2048), 8), ((1, 900, 255), 5),
          ((1, 300, 4099), 1), ((700, 1, 2048), 8)]


def betas(n, dtype):
    far = np.concatenate([np.linspace(-130, -80, 201), np.linspace(-20, 20, 41), -np.geomspace(1, MOST[dtype], 80),
                          np.geomspace(1, MOST[dtype], 40), [-0.0, 0.0]])
    return torch.from_numpy(np.resize(far, n)).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_silu_far_out(lib, dtype, shape, groups):
    n, s, c = shape
    b = betas(c, dtype)
    g = torch.Generator().manual_seed(sum(shape))
    x = torch.randn(shape, generator=g).to(DT[dtype]).cuda()
    gamma = torch.zeros(c, dtype=DT[dtype], device="cuda")
    y, mean, inv = lib.ep_group_norm(x, gamma, b.cuda(), groups, activation=lib.EP_ACT_SILU, mean=True, inv_std_dev=True)
    dy = torch.zeros_like(x)
    dy[0, 0] = 1.0
    dx, dg, db = lib.ep_group_norm_grad(dy, x, gamma, b.cuda(), mean, inv, groups, lib.EP_ACT_SILU)
    u = b.double().numpy()
    with np.errstate(over="ignore"):
        sig = 1.0 / (1.0 + np.exp(-u))
    silu, slope = u * sig, sig * (1.0 + u * (1.0 - sig))
    rel = (8 if dtype == "f32" else 16 + np.minimum(np.abs(u), 100)) * U32
    tiny = 2.0 ** -116   # |u| <= 130 times 2^-123
    delta = rel * np.abs(silu) + tiny
    assert_within(y.reshape(-1, c)[:: max(1, n * s // 7)].cpu(), np.broadcast_to(silu, (len(range(0, n * s, max(1, n * s // 7))), c)),
                  delta, "silu")
    assert_within(db.cpu(), slope, rel * sig * (1 + np.minimum(np.abs(u), 20)) + tiny, "silu slope")
    assert bool(torch.isfinite(dx).all())
