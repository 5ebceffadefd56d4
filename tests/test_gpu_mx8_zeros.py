"""The RMS norm to MX8 where values are 0 or small beside a large 1 / root mean square: rows and
groups of zeros, padding, gamma's zeros, NaN and infinities, and a padded batch through a block."""
import numpy as np
import pytest
import torch

from oracle import products as op
from tests._helpers import U32
from tests._products import DT, assert_mx8, assert_within, at_offset, cuda, f64, mx8_f64, scale_bytes, y_delta, z_delta
from tests.test_gpu_mx8_chain import block_inputs, run_block

pytestmark = pytest.mark.gpu

# one element, one group, a group and one, several to a warp, ragged, several warps, and rows too long for the registers
WIDTHS = [1, 3, 32, 33, 35, 64, 77, 200, 512, 1001, 4096, 4100, 8192, 16384, 16392]


def zero_rows(h, dtype, seed):
    """Rows of zeros, rows of root mean square 1e-6 to 1, and rows with groups, ends or all but one element of 0."""
    g = torch.Generator().manual_seed(seed)
    stds = [0.0, 1e-6, 1e-5, 1e-4, 1e-3, 0.01, 0.03, 0.1, 0.2, 0.25, 1.0]
    x = torch.stack([torch.randn(h, generator=g) * s for s in stds] * 2)
    n = len(stds)
    last = (h - 1) // 32 * 32
    x[n:, : min(32, max(1, h // 2))] = 0          # the first group (or some of it)
    if h > 64:
        x[n + 3, 32:64] = 0
    x[n + 5:, last:] = 0                          # the last group, whole or of a few elements
    one = torch.zeros(4, h)
    one[0, 0] = one[1, -1] = 1e-3
    one[2, h // 2] = -0.2
    one[3] = -0.0
    return torch.cat([x, one]).to(DT[dtype])


def check_norm(lib, x, g, eps, off=0):
    dx, dg = (at_offset(t, off) if off else t for t in cuda(x, g))
    q, s, su, inv = lib.ep_skip_rms_norm_mx8(dx, None, dg, epsilon=eps, input_skip_bias_sum=True, inv_std_dev=True)
    assert torch.equal(su.cpu(), x)
    o = op.rms_norm(f64(x), None, f64(g), None, eps)
    # s is exact; inv as in test_gpu_mx8.py: 64 u; y: two products, and the one before them
    assert_within(inv, o["inv"], 64 * U32 * o["inv"], "rms inv zeros")
    assert_mx8(q, s, o["y"], 68 * U32 * np.abs(o["y"]), "rms q zeros")
    zero = o["y"] == 0
    assert (f64(q.float())[zero] == 0).all()
    b = scale_bytes(s)
    empty = op.mx8_group_max(o["y"]) == 0
    assert empty.any() and (b[empty] == 1).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("h", WIDTHS)
def test_zero_rows_and_groups(lib, h, dtype):
    g = (torch.randn(h, generator=torch.Generator().manual_seed(52)) * 0.2 + 1).to(DT[dtype])
    x = zero_rows(h, dtype, 51)
    for eps in (lib.DEFAULT_EPSILON, 1e-5):
        check_norm(lib, x, g, eps)
    check_norm(lib, x, g, 1e-6, off=1)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("h", [33, 77, 200, 1001, 4096, 16392])
def test_zeros_of_gamma(lib, h, dtype):
    """Groups that gamma makes 0, and values that it makes as small as the scale's limits."""
    g = (torch.randn(h, generator=torch.Generator().manual_seed(54)) * 0.2 + 1).to(DT[dtype])
    g[:32] = 0
    g[-1:] = 0
    if h > 128:
        g[64:128] = 0
    x = zero_rows(h, dtype, 53)
    check_norm(lib, x, g, lib.DEFAULT_EPSILON)
    if dtype != "f16":
        g[32:64] = 2.0 ** -120
        check_norm(lib, x, g, lib.DEFAULT_EPSILON)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("h", [1, 7, 40, 77, 768, 4104, 20001])
def test_skip_that_cancels(lib, h, dtype):
    """input + skip = 0: the row is 0 and its statistic 1 / sqrt(epsilon)."""
    x = torch.randn(5, h, generator=torch.Generator().manual_seed(55)).to(DT[dtype]).cuda()
    g = torch.ones(h, dtype=DT[dtype], device="cuda")
    q, s, su, inv = lib.ep_skip_rms_norm_mx8(x, -x, g, input_skip_bias_sum=True, inv_std_dev=True)
    assert not su.any() and not q.float().any() and (s.view(torch.uint8) == 1).all()
    assert_within(inv, np.full((5, 1), 1 / np.sqrt(float(np.float32(lib.DEFAULT_EPSILON)))), 64 * U32 * 1e6, "rms inv zeros")


@pytest.mark.parametrize("h", [5, 40, 77, 768, 16392, 20001])
def test_not_finite(lib, h):
    """A NaN makes its row NaN; an infinity itself, beside zeros (its row's statistic is 0); 1 / sqrt(0) of a row of zeros
    infinite, and the row NaN.  The scales are those of the other values."""
    x = torch.randn(4, h, generator=torch.Generator().manual_seed(56))
    x[0, 3], x[1, 4], x[2] = float("nan"), float("inf"), 0.0
    g = torch.ones(h, device="cuda")
    q, s = lib.ep_skip_rms_norm_mx8(x.cuda(), None, g, epsilon=0.0)[:2]
    got, b = q.float().cpu(), scale_bytes(s)
    assert got[0].isnan().all() and got[2].isnan().all()
    assert got[1, 4].isnan() and not got[1, :4].any() and not got[1, 5:].any()
    assert (b[:3] == 1).all()
    assert got[3].isfinite().all()


def test_padded_batch_through_a_block(lib):
    """Tokens of zeros among others, their activations kept in 8 bits: every gradient is the oracle's."""
    rows, hidden, inner = 150, 256, 328
    p = block_inputs(rows, hidden, inner, "bf16", 57)
    pad = torch.arange(rows, device="cuda") % 5 > 2
    for name in ("x", "skip", "dy"):
        p[name][pad] = 0
    o = run_block(lib, p)
    assert (f64(o["q"][0].float())[pad.cpu().numpy()] == 0).all()
    for name, v in o.items():
        for t in v if isinstance(v, tuple) else (v,):
            if t.dtype != torch.float8_e8m0fnu:
                assert torch.isfinite(t.float()).all(), name
    half, slope = 2.0 ** -8, 64 * U32
    w1, a, h = mx8_f64(*o["w1"]), mx8_f64(*o["q"]), mx8_f64(*o["hq"])
    m1 = op.matmul(a, w1, f64(p["b1"]), None, "quick_gelu")
    d1 = z_delta(hidden, m1["z_scale"])
    assert_within(o["h"], m1["y"], y_delta(m1["z"], m1["y"], d1, "quick_gelu", 1.702), "block h")
    g2 = op.matmul_grad(f64(p["dy"]), h, f64(p["w2"]))
    assert_within(o["dw2"], g2["dW"], z_delta(rows, g2["dW_scale"]), "block dw2")
    g1 = op.matmul_grad(f64(o["dh"]), a, f64(p["w1"]), mx8_f64(*o["z"]), "quick_gelu")
    assert_within(o["dw1"], g1["dW"], (half + slope) * g1["dW_scale"] + z_delta(rows, g1["dW_scale"]), "block dw1")
    gn = op.rms_norm_grad(f64(o["dn"]), f64(o["total"]), f64(p["gamma"]), f64(o["inv"]), f64(p["dy"]))
    assert_within(o["dx"], gn["dX"], 64 * U32 * gn["dX_scale"], "block dx")
    assert_within(o["dg"], gn["dgamma"], 128 * U32 * gn["dgamma_scale"], "block dgamma")
