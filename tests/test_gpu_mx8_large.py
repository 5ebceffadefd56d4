"""MX8 rows, the RMS norm and the matrix product past 2^31 elements, and long sums."""
import numpy as np
import pytest
import torch

from oracle import products as op
from tests._helpers import U32
from tests._products import HALF, assert_mx8, assert_within, f64, mx8_f64, z_delta

pytestmark = pytest.mark.gpu


def some_rows(rows):
    return torch.tensor([0, 1, rows // 3, rows // 2 + 1, rows - 2, rows - 1], device="cuda")


@pytest.mark.parametrize("h", [4096, 4097])
def test_rows_past_2_31(lib, h):
    rows = (1 << 31) // h + 1000
    g = torch.Generator(device="cuda").manual_seed(41)
    x = torch.empty(rows, h, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    at = some_rows(rows)
    q, s = lib.ep_quantize_mx8(x)
    wq, wb = op.mx8_quantize(f64(x[at]))
    np.testing.assert_array_equal(mx8_f64(q[at], s[at]), op.mx8_values(wq, wb))
    y = lib.ep_dequantize_mx8(q, s, torch.bfloat16)
    np.testing.assert_array_equal(f64(y[at]), op.mx8_values(wq, wb))
    del y
    gamma = (torch.rand(h, device="cuda", generator=g) + 0.5).bfloat16()
    q, s, total, inv = lib.ep_skip_rms_norm_mx8(x, None, gamma, Q=q, scales=s, input_skip_bias_sum=True, inv_std_dev=True)
    o = op.rms_norm(f64(x[at]), None, f64(gamma), None, lib.DEFAULT_EPSILON)
    assert torch.equal(total[at], x[at])
    assert_mx8(q[at], s[at], o["y"], 100 * U32 * np.abs(o["y"]), "rms q large")
    dx, dg, _ = lib.ep_skip_rms_norm_grad(total, x, gamma, inv, dX=total)
    d = op.rms_norm_grad(f64(x[at]), f64(x[at]), f64(gamma), f64(inv[at]))
    assert_within(dx[at], d["dX"], 64 * U32 * d["dX_scale"], "rms dX large")
    # every term of dgamma is x^2 inv, positive: the float32 sum's depth (rows a block, then blocks) is below 2000
    want = torch.zeros(h, dtype=torch.float64, device="cuda")
    for r in range(0, rows, 1 << 16):
        p = x[r:r + (1 << 16)].double()
        want += (p * p * inv[r:r + (1 << 16)]).sum(0)
    w = want.cpu().numpy()
    assert_within(dg, w, 2000 * U32 * w, "rms dgamma large")


@pytest.mark.parametrize("m,n", [(70000, 40000), (70001, 39999), (33, 1 << 26)])
def test_products_past_2_31(lib, m, n):
    k = 64
    g = torch.Generator(device="cuda").manual_seed(42)
    a = torch.empty(m, k, dtype=torch.float16, device="cuda").normal_(generator=g)
    w = torch.empty(n, k, dtype=torch.float16, device="cuda").normal_(generator=g) / 8
    b = torch.empty(n, dtype=torch.float16, device="cuda").normal_(generator=g)
    y, z, _ = lib.ep_matmul_bias_act(a, w, b, Z=True)
    rows, cols = some_rows(m), some_rows(n)
    o = op.matmul(f64(a[rows]), f64(w[cols]), f64(b[cols]))
    for t in (y, z):
        assert_within(t[rows][:, cols], o["z"], z_delta(k, o["z_scale"]), "mm large")
    del z
    _, q, s = lib.ep_matmul_bias_act(a, w, b, Y=y, Z=torch.float8_e4m3fn)
    c = int(cols[-1]) // 32 * 32
    tail = op.matmul(f64(a[rows]), f64(w[c:]), f64(b[c:]))
    assert_mx8(q[rows][:, c:].contiguous(), s[rows][:, c // 32:].contiguous(), tail["z"], z_delta(k, tail["z_scale"]), "mm z8 large")
    if m * n < 1 << 31 or n > 1 << 20:
        return
    # the gradient: dz has 2^31 elements too; depths of 70000 and 40000
    dy = y
    da, dw, db = lib.ep_matmul_bias_act_grad(dy, a, w, dy, lib.EP_ACT_RELU, dbias=True)
    part = torch.relu(dy[rows].float()).double()
    want = part @ w.double()
    scale = part.abs() @ w.double().abs()
    assert_within(da[rows], want.cpu().numpy(), z_delta(n, scale.cpu().numpy()), "mm dA large")
    part = torch.relu(dy[:, cols].float()).double()
    want, scale = part.t() @ a.double(), part.abs().t() @ a.double().abs()
    assert_within(dw[cols], want.cpu().numpy(), z_delta(m, scale.cpu().numpy()), "mm dW large")
    # float32 sums of positive terms, the depth below 1500; from 65520 on a float16 result is infinite
    want, delta = part.sum(0).cpu().numpy(), 1500 * U32 * part.abs().sum(0).cpu().numpy()
    assert (np.abs(want - 65520) > delta).all()
    assert_within(db[cols], np.where(want > 65520, np.inf, want), delta, "mm dbias large")


@pytest.mark.parametrize("mx8", [False, True])
def test_long_sums(lib, mx8):
    m, n, k = 5, 40, 300000
    g = torch.Generator(device="cuda").manual_seed(43)
    a = torch.empty(m, k, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.empty(n, k, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    if mx8:
        (qa, sa), (qw, sw) = lib.ep_quantize_mx8(a), lib.ep_quantize_mx8(w)
        y = lib.ep_matmul_bias_act(qa, qw, A_scales=sa, W_scales=sw, dtype=torch.bfloat16)[0]
        o = op.matmul(mx8_f64(qa, sa), mx8_f64(qw, sw))
    else:
        y = lib.ep_matmul_bias_act(a, w)[0]
        o = op.matmul(f64(a), f64(w))
    assert_within(y, o["y"], z_delta(k, o["z_scale"]), "mm long")
    assert HALF[torch.bfloat16] == 2.0 ** -8
