"""Pins of the GroupNorm / BiasDropout oracle: published words of the generator,
hand-worked groups, invariants, and differences against its gradients (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import training as tr


@pytest.mark.parametrize("counter,key,want", [
    # the known answers published with the generator
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_known_answers(counter, key, want):
    assert tuple(tr.philox4x32(counter, key)) == want


def test_words_follow_the_counter_layout():
    seed, offset = 0xA4093822_00000007, 0x0370734413198A2E
    for first in (0, 4, (1 << 34) + 8):   # blocks beyond 32 bits use the counter's second word
        words = tr.dropout_words(11, seed, offset, first)
        for i in (0, 3, 4, 10):
            block = (first + i) // 4
            want = tr.philox4x32((block & 0xFFFFFFFF, block >> 32, offset & 0xFFFFFFFF, offset >> 32),
                                 (seed & 0xFFFFFFFF, seed >> 32))[(first + i) % 4]
            assert int(words[i]) == want


def test_keep_rate_and_limits():
    n = 1 << 16
    for ratio in (0.1, 0.5, 0.9):
        rate = tr.dropout_keep(n, ratio, 5, 9).mean()
        # five standard deviations of a binomial share
        assert abs(rate - (1 - ratio)) < 5 * np.sqrt(ratio * (1 - ratio) / n)
    assert tr.dropout_keep(n, 0.0, 5, 9).all()
    assert not np.array_equal(tr.dropout_keep(n, 0.5, 5, 9), tr.dropout_keep(n, 0.5, 5, 10))
    assert not np.array_equal(tr.dropout_keep(n, 0.5, 5, 9), tr.dropout_keep(n, 0.5, 6, 9))


def test_bias_dropout_by_hand():
    x, b, r = np.array([[1.0, 2.0], [3.0, 4.0]]), np.array([0.5, -1.0]), np.full((2, 2), 10.0)
    d = tr.bias_dropout(x, 0.75, 1, 2, bias=b, residual=r)
    want = np.where(d["keep"], (x + b) * 4.0, 0.0) + 10.0
    assert np.array_equal(d["Y"], want)
    g = tr.bias_dropout_grad(np.ones((2, 2)), 0.75, 1, 2)
    assert np.array_equal(g["keep"], d["keep"]) and np.array_equal(g["dbias"], g["dX"].sum(0))


def test_group_norm_by_hand():
    # one sample, two positions, two groups of two channels: {1, 2, 3, 4} and {0, 0, 2, 2}
    x = np.array([[[1.0, 2.0, 0.0, 0.0], [3.0, 4.0, 2.0, 2.0]]])
    d = tr.group_norm(x, np.ones(4), np.zeros(4), 2, 0.0)
    s = np.sqrt(1.25)
    assert np.allclose(d["mean"], [[2.5, 1.0]]) and np.allclose(d["inv_std_dev"], [[1 / s, 1.0]])
    assert np.allclose(d["Y"][0], [[-1.5 / s, -0.5 / s, -1, -1], [0.5 / s, 1.5 / s, 1, 1]])


def test_group_norm_special_cases():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(3, 5, 7, 12, generator=g, dtype=torch.float64)   # (N, H, W, C)
    gamma, beta = torch.randn(12, generator=g, dtype=torch.float64), torch.randn(12, generator=g, dtype=torch.float64)
    eps = float(np.float32(1e-3))
    for groups in (1, 3, 12):
        want = torch.nn.functional.group_norm(x.permute(0, 3, 1, 2), groups, gamma, beta, eps)
        want = torch.nn.functional.silu(want).permute(0, 2, 3, 1)
        got = tr.group_norm(x, gamma, beta, groups, 1e-3, silu=True)["Y"]
        assert np.allclose(got, want.numpy(), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("with_beta", [False, True])
def test_group_norm_grad_is_the_derivative(silu, with_beta):
    g = np.random.default_rng(7)
    x = g.normal(size=(2, 3, 6))
    gamma, beta = g.normal(size=6), g.normal(size=6) if with_beta else None
    w = g.normal(size=x.shape)

    def value(x, gamma, beta):
        return float((tr.group_norm(x, gamma, beta, 2, 1e-2, silu)["Y"] * w).sum())

    f = tr.group_norm(x, gamma, beta, 2, 1e-2, silu)
    d = tr.group_norm_grad(w, x, gamma, beta, f["mean"], f["inv_std_dev"], 2, silu)
    step = 1e-5   # central differences of a smooth function: step^2 away
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = step
        assert abs((value(x + e, gamma, beta) - value(x - e, gamma, beta)) / (2 * step) - d["dX"][i]) < 1e-7
    for c in range(6):
        e = np.zeros(6)
        e[c] = step
        assert abs((value(x, gamma + e, beta) - value(x, gamma - e, beta)) / (2 * step) - d["dgamma"][c]) < 1e-7
        if with_beta:
            assert abs((value(x, gamma, beta + e) - value(x, gamma, beta - e)) / (2 * step) - d["dbeta"][c]) < 1e-7
