"""Products of values at the ends of their types: NaN and infinities in either operand, subnormals, scales far apart,
each against float64 on small and on many tiles."""
import numpy as np
import pytest
import torch

from oracle import products as op
from tests._helpers import U32
from tests._products import DT, assert_within, f64, mx8_f64, product_inputs, cuda, z_delta

pytestmark = pytest.mark.gpu

SHAPES = [(3, 72, 96), (40, 130, 200), (300, 264, 77), (1040, 2568, 64)]


def check(y, a64, w64, b64):
    with np.errstate(invalid="ignore"):
        z, scale = a64 @ w64.T + b64, np.abs(a64) @ np.abs(w64).T + np.abs(b64)
    fin = np.isfinite(scale)
    assert_within(y, z, np.where(fin, z_delta(a64.shape[1], np.where(fin, scale, 0)), 0), "mm values")


@pytest.mark.parametrize("mnk", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("off", [0, 1])
def test_not_finite(lib, mnk, dtype, off):
    """An infinity or NaN reaches its own row or column alone, at the ends of rows, tiles and K too."""
    m, n, k = mnk
    a, w, b, _ = product_inputs(m, n, k, dtype, 71)
    a[0, 0], a[m - 1, k - 1], a[m // 2, k // 2] = float("inf"), float("-inf"), float("nan")
    w[n - 1, 0], w[1, k - 1] = float("inf"), float("nan")
    b[n // 2] = float("-inf")
    if off:
        a, w = (torch.cat([t.view(-1)[:1], t.view(-1)])[1:].view(t.shape) for t in (a, w))
    y = lib.ep_matmul_bias_act(*cuda(a, w, b))[0]
    check(y, f64(a), f64(w), f64(b))


@pytest.mark.parametrize("mnk", SHAPES, ids=str)
def test_mx8_not_finite(lib, mnk):
    """E4M3 NaN and groups whose scale is NaN (made of an infinity), in A and in W."""
    m, n, k = mnk
    a, w, b, _ = product_inputs(m, n, k, "bf16", 72)
    a[0, 0], a[m - 1, k - 1], w[n - 1, k // 2], w[1, 0] = float("nan"), float("inf"), float("nan"), float("-inf")
    (qa, sa), (qw, sw) = lib.ep_quantize_mx8(a.cuda()), lib.ep_quantize_mx8(w.cuda())
    a64, w64 = mx8_f64(qa, sa), mx8_f64(qw, sw)
    y = lib.ep_matmul_bias_act(qa, qw, b.cuda(), A_scales=sa, W_scales=sw, dtype=torch.bfloat16)[0]
    assert np.isnan(a64).any(1).sum() == 2 and np.isnan(w64).any(1).sum() == 2
    check(y, a64, w64, f64(b))


@pytest.mark.parametrize("mnk", SHAPES, ids=str)
@pytest.mark.parametrize("ea,ew", [(100, -100), (-110, 112), (60, 50), (-60, -55), (0, -120)])
def test_mx8_scales_far_apart(lib, mnk, ea, ew):
    """Rows of any magnitude: scales multiply without a limit of their own (bfloat16 results reach 2^128)."""
    m, n, k = mnk
    a, w, _, _ = product_inputs(m, n, k, "bf16", 73)
    a, w = (a.float() * 2.0 ** ea).bfloat16(), (w.float() * 2.0 ** ew).bfloat16()
    (qa, sa), (qw, sw) = lib.ep_quantize_mx8(a.cuda()), lib.ep_quantize_mx8(w.cuda())
    y = lib.ep_matmul_bias_act(qa, qw, A_scales=sa, W_scales=sw, dtype=torch.bfloat16)[0]
    check(y, mx8_f64(qa, sa), mx8_f64(qw, sw), np.zeros(n))


@pytest.mark.parametrize("mnk", SHAPES, ids=str)
@pytest.mark.parametrize("dtype,ea,ew", [("f16", -18, 8), ("f16", -20, 0), ("bf16", -127, 100), ("bf16", -60, -50), ("bf16", 60, 55)])
def test_subnormal_and_far_operands(lib, mnk, dtype, ea, ew):
    m, n, k = mnk
    a, w, _, _ = product_inputs(m, n, k, dtype, 74)
    a, w = (a.double() * 2.0 ** ea).to(DT[dtype]), (w.double() * 2.0 ** ew).to(DT[dtype])
    y = lib.ep_matmul_bias_act(*cuda(a, w))[0]
    check(y, f64(a), f64(w), np.zeros(n))
    dy = torch.ones(m, n, dtype=DT[dtype], device="cuda")
    da, dw, _ = lib.ep_matmul_bias_act_grad(dy, *cuda(a, w))
    o = op.matmul_grad(f64(dy), f64(a), f64(w))
    assert_within(da, o["dA"], z_delta(n, o["dA_scale"]), "mm values dA")
    assert_within(dw, o["dW"], z_delta(m, o["dW_scale"]), "mm values dW")


@pytest.mark.parametrize("rank", [1, 3, 4])
def test_rows_of_any_rank(lib, rank):
    """(H,), (a, b, H) and (a, b, c, H): the outputs and the statistic have the rows' dimensions."""
    shape = (3, 2, 5, 72)[4 - rank:]
    g = torch.Generator(device="cuda").manual_seed(75)
    x, dy = (torch.randn(shape, device="cuda", generator=g).half() for _ in range(2))
    gamma = torch.ones(72, device="cuda").half()
    q, s, su, inv = lib.ep_skip_rms_norm_mx8(x, None, gamma, input_skip_bias_sum=True, inv_std_dev=True)
    assert q.shape == x.shape and s.shape == shape[:-1] + (3,) and inv.shape == shape[:-1] + (1,) and torch.equal(su, x)
    dx, dg, _ = lib.ep_skip_rms_norm_grad(dy, su, gamma, inv)
    flat = lib.ep_skip_rms_norm_grad(dy.view(-1, 72), su.view(-1, 72), gamma, inv.view(-1, 1))
    assert torch.equal(dx.view(-1, 72), flat[0]) and torch.equal(dg, flat[1])
    o = op.rms_norm_grad(f64(dy).reshape(-1, 72), f64(x).reshape(-1, 72), np.ones(72), f64(inv).reshape(-1, 1))
    assert_within(dx, o["dX"], 64 * U32 * o["dX_scale"], "rms dX rank")
