"""Pins of the MX8, RMS norm and matrix product oracle: torch's own 8-bit conversions,
closed values, torch's float64 functions, and differences for the gradients."""
import math

import numpy as np
import pytest
import torch

from oracle import products as op


def test_e4m3_is_torch_s():
    x = torch.cat([torch.linspace(-448, 448, 40001, dtype=torch.float64), torch.linspace(-0.05, 0.05, 20001, dtype=torch.float64)])
    x = x.float()  # torch rounds float32
    want = x.to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(op.e4m3_round(x.double().numpy()), want)


def test_ties_go_to_even():
    np.testing.assert_array_equal(op.e4m3_round(np.array([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 1.0625, 1.1875])),
                                  [16.0, 20.0, 0.0, 2.0 ** -8, 1.0, 1.25])


def test_scales_are_the_smallest_powers():
    a = np.concatenate([[448.0, 448.0001, 449.0, 224.0, 224.1, 1.0, 1.75, 1.76, 2.0 ** -118, 2.0 ** -126, 0.0], 2.0 ** np.arange(-110.0, 127)])
    b = op.mx8_bytes(a)
    k = 2.0 ** (b - 127.0)
    assert (a <= 448 * k).all()
    inner = b > 1
    assert (a[inner] > 224 * k[inner]).all()
    assert op.mx8_bytes(np.array([np.inf])) == 255 and op.mx8_bytes(np.array([0.0])) == 1


def test_rows_and_groups():
    x = np.zeros((2, 70))
    x[0, 3], x[0, 40], x[0, 69], x[1, 31], x[1, 32] = 448.0, -1.0, 2.0, 896.0, 3.0
    q, b = op.mx8_quantize(x)
    np.testing.assert_array_equal(b, [[127, 119, 120], [128, 120, 1]])
    np.testing.assert_array_equal(op.mx8_values(q, b), x)
    assert q[0, 40] == -256.0 and q[1, 31] == 448.0


def test_norm_and_its_gradient():
    g = np.random.default_rng(3)
    x, skip, gamma, bias, w, v = (g.normal(size=d) for d in ((3, 5), (3, 5), 5, 5, (3, 5), (3, 5)))
    o = op.rms_norm(x, skip, gamma, bias, 1e-3)
    s = torch.tensor(x + skip + bias, requires_grad=True)
    gt, bt = torch.tensor(gamma, requires_grad=True), torch.zeros(5, dtype=torch.float64, requires_grad=True)
    t = s + bt
    y = t * torch.rsqrt((t * t).mean(1, keepdim=True) + float(np.float32(1e-3))) * gt
    assert np.allclose(o["y"], y.detach().numpy(), rtol=1e-13, atol=0)
    ((y * torch.tensor(w)).sum() + (t * torch.tensor(v)).sum()).backward()
    d = op.rms_norm_grad(w, o["s"], gamma, o["inv"], v)
    assert np.allclose(d["dX"], s.grad.numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(d["dgamma"], gt.grad.numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(d["dbias"], bt.grad.numpy(), rtol=1e-12, atol=1e-13)
    assert (d["dX_scale"] >= np.abs(d["dX"]) * (1 - 1e-12)).all() and (d["dgamma_scale"] >= np.abs(d["dgamma"]) * (1 - 1e-12)).all()


@pytest.mark.parametrize("act", op.ACTS)
def test_activations_are_torch_s(act):
    z = torch.linspace(-9, 9, 1001, dtype=torch.float64, requires_grad=True)
    F = torch.nn.functional
    y = {"none": lambda: z * 1, "silu": lambda: F.silu(z), "relu": lambda: F.relu(z), "gelu": lambda: F.gelu(z),
         "fast_gelu": lambda: F.gelu(z, approximate="tanh"), "quick_gelu": lambda: z * torch.sigmoid(float(np.float32(0.9)) * z)}[act]()
    assert np.allclose(op.activation(z.detach().numpy(), act, 0.9), y.detach().numpy(), rtol=1e-11, atol=1e-13)
    y.sum().backward()
    got = op.activation_slope(z.detach().numpy(), act, 0.9)
    keep = np.abs(z.detach().numpy()) > 1e-9  # (relu's corner)
    assert np.allclose(got[keep], z.grad.numpy()[keep], rtol=1e-9, atol=1e-12)
    step = 1e-5
    zz = z.detach().numpy()[keep]
    diff = (op.activation(zz + step, act, 0.9) - op.activation(zz - step, act, 0.9)) / (2 * step)
    assert np.abs(diff - got[keep])[np.abs(zz) > 2 * step].max() < 1e-8


@pytest.mark.parametrize("act", op.ACTS)
def test_limits(act):
    y = op.activation(np.array([-np.inf, 0.0, np.inf]), act)
    np.testing.assert_array_equal(y, [0.0 if act != "none" else -np.inf, 0.0, np.inf])
    assert math.isnan(op.activation(np.array([np.nan]), act)[0])


@pytest.mark.parametrize("act", op.ACTS)
def test_product_gradient_by_differences(act):
    g = np.random.default_rng(5)
    a, w, b, v = (g.normal(size=d) for d in ((3, 4), (5, 4), 5, (3, 5)))

    def value(a, w, b):
        return float((op.matmul(a, w, b, None, act)["y"] * v).sum())

    d = op.matmul_grad(v, a, w, op.matmul(a, w, b)["z"], act)
    step = 1e-5
    for arr, name, at in ((a, "dA", 0), (w, "dW", 1), (b, "dbias", 2)):
        for i in np.ndindex(arr.shape):
            e = np.zeros_like(arr)
            e[i] = step
            args = [a, w, b]
            hi, lo = list(args), list(args)
            hi[at], lo[at] = arr + e, arr - e
            assert abs((value(*hi) - value(*lo)) / (2 * step) - d[name][i]) < 1e-7
    assert (d["dA_scale"] >= np.abs(d["dA"]) - 1e-12).all() and (d["dW_scale"] >= np.abs(d["dW"]) - 1e-12).all()


def test_product_residual_and_terms():
    a, w = np.array([[1.0, -2.0]]), np.array([[3.0, 4.0], [0.5, 0.25]])
    o = op.matmul(a, w, np.array([1.0, -1.0]), np.array([[10.0, 20.0]]), "relu")
    np.testing.assert_array_equal(o["z"], [[-4.0, -1.0]])
    np.testing.assert_array_equal(o["y"], [[10.0, 20.0]])
    np.testing.assert_array_equal(o["z_scale"], [[12.0, 2.0]])
