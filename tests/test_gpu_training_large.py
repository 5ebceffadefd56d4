"""GroupNorm and BiasDropout on tensors past 2^31 elements: every offset must be
computed in 64 bits.  Inputs are drawn on the device; sums are checked against
float64 sums taken there, results on sampled rows on both sides of element 2^31."""
import numpy as np
import pytest
import torch

from gen import synth
from oracle import training as tr
from tests._helpers import U32
from tests._training import assert_within

pytestmark = pytest.mark.gpu

E31 = 1 << 31
EPS = 1e-5


@pytest.fixture(autouse=True)
def _release_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def rows_to_check(n_rows, row_len):
    r31 = E31 // row_len
    picks = set(range(0, n_rows, n_rows // 13)) | {0, 1, n_rows - 2, n_rows - 1}
    return torch.tensor(sorted(picks | set(range(r31 - 2, r31 + 3))), dtype=torch.int64, device="cuda")


def chunked(rows, f, step=1 << 18):
    """Sum of f(a, b) over row ranges, in float64."""
    total = 0
    for a in range(0, rows, step):
        total = total + f(a, min(rows, a + step))
    return total


@pytest.mark.parametrize("C,groups", [(256, 4), (189, 9)])
def test_group_norm_one_sample_past_2_31_elements(lib, C, groups):
    S, D = E31 // C + 513, C // groups
    x = synth.device_normal((1, S, C), "f16", seed=71)
    dy = synth.device_normal((1, S, C), "f16", seed=72)
    gamma = synth.device_normal((C,), "f16", seed=73, std=0.2) + 1
    beta = synth.device_normal((C,), "f16", seed=74, std=0.2)
    y, mean, inv = lib.ep_group_norm(x, gamma, beta, groups, EPS, mean=True, inv_std_dev=True)
    by_group = lambda t, a, b: t[0, a:b].double().view(b - a, groups, D)   # noqa: E731
    m = chunked(S, lambda a, b: by_group(x, a, b).sum((0, 2))) / (S * D)
    v = chunked(S, lambda a, b: ((by_group(x, a, b) - m[:, None]) ** 2).sum((0, 2))) / (S * D)
    r = 1 / torch.sqrt(v + EPS)
    assert_within(mean[0].cpu(), m.cpu().numpy(), 16 * U32 * (m.abs().cpu().numpy() + 1), "gn mean")
    assert_within(inv[0].cpu(), r.cpu().numpy(), 64 * U32 * r.cpu().numpy(), "gn inv")
    rows = rows_to_check(S, C)
    ga, be = (t.double().cpu().numpy() for t in (gamma, beta))
    mc, rc = (np.repeat(t.cpu().numpy(), D) for t in (m, r))
    h = (x[0, rows].double().cpu().numpy() - mc) * rc
    scale = np.abs(h) + np.abs(mc * rc)
    assert_within(y[0, rows].cpu(), h * ga + be, 64 * U32 * (scale * np.abs(ga) + np.abs(be)), "gn")

    # the gradient, from the statistics of the forward call
    del y
    mu, ri = (t[0].double() for t in (mean, inv))
    gd = gamma.double().view(groups, D)

    def terms(a, b):
        du, hh = by_group(dy, a, b), (by_group(x, a, b) - mu[:, None]) * ri[:, None]
        w = du * gd
        return torch.stack([du.sum(0), (du * hh).sum(0), du.abs().sum(0), (du * hh).abs().sum(0),
                            w.sum((0, 2))[:, None].expand(groups, D), (w * hh).sum((0, 2))[:, None].expand(groups, D)])
    db, dg, db_abs, dg_abs, m1, m2 = chunked(S, terms)
    m1, m2 = m1 / (S * D), m2 / (S * D)
    dx, dgamma, dbeta = lib.ep_group_norm_grad(dy, x, gamma, beta, mean, inv, groups)
    flat = lambda t: t.reshape(-1).cpu().numpy()   # noqa: E731
    assert_within(dbeta.cpu(), flat(db), 64 * U32 * flat(db_abs), "gn dbeta")
    assert_within(dgamma.cpu(), flat(dg), 64 * U32 * flat(dg_abs), "gn dgamma")
    w = dy[0, rows].double().cpu().numpy() * ga
    mu, ri = (np.repeat(t.cpu().numpy(), D) for t in (mu, ri))
    h = (x[0, rows].double().cpu().numpy() - mu) * ri
    want = ri * (w - flat(m1) - h * flat(m2))
    size = ri * (np.abs(w) + 1 + (np.abs(h) + np.abs(mu * ri)))
    assert_within(dx[0, rows].cpu(), want, 64 * U32 * size, "gn dX")


def test_group_norm_tokens_past_2_31_elements(lib):
    C, groups = 4096, 32
    N = E31 // C + 77
    x = synth.device_normal((N, 1, C), "f16", seed=75)
    dy = synth.device_normal((N, 1, C), "f16", seed=76)
    gamma = synth.device_normal((C,), "f16", seed=77, std=0.2) + 1
    beta = synth.device_normal((C,), "f16", seed=78, std=0.2)
    y, mean, inv = lib.ep_group_norm(x, gamma, beta, groups, EPS, mean=True, inv_std_dev=True)
    dx, dgamma, dbeta = lib.ep_group_norm_grad(dy, x, gamma, beta, mean, inv, groups)
    rows = rows_to_check(N, C)
    o = tr.group_norm(x[rows].cpu(), gamma.cpu(), beta.cpu(), groups, EPS)
    assert_within(mean[rows].cpu(), o["mean"], 16 * U32 * (np.abs(o["mean"]) + 1), "gn mean")
    assert_within(inv[rows].cpu(), o["inv_std_dev"], 64 * U32 * o["inv_std_dev"], "gn inv")
    assert_within(y[rows].cpu(), o["Y"].reshape(rows.numel(), 1, C),
                  64 * U32 * (np.abs(o["Y"].reshape(rows.numel(), 1, C)) + 8), "gn")
    o = tr.group_norm_grad(dy[rows].cpu(), x[rows].cpu(), gamma.cpu(), beta.cpu(), mean[rows].cpu(), inv[rows].cpu(),
                           groups)
    assert_within(dx[rows].cpu(), o["dX"], 64 * U32 * o["dX_scale"], "gn dX")
    db = chunked(N, lambda a, b: torch.stack([dy[a:b, 0].double().sum(0), dy[a:b, 0].double().abs().sum(0)]), 1 << 14)
    assert_within(dbeta.cpu(), db[0].cpu().numpy(), 64 * U32 * db[1].cpu().numpy(), "gn dbeta")
    assert bool(torch.isfinite(dgamma).all())


def test_bias_dropout_past_2_31_elements(lib):
    C, seed, offset, ratio = 4104, 0x1234567_89ABCDEF, 0xFEDCBA98_00000003, 0.5
    R = E31 // C + 1001
    x = synth.device_normal((R, C), "f16", seed=79)
    b = synth.device_normal((C,), "f16", seed=80, std=0.1)
    r = synth.device_normal((R, C), "f16", seed=81)
    y = lib.ep_bias_dropout(x, ratio, seed, offset, bias=b, residual=r)
    dx, dbias = lib.ep_bias_dropout_grad(x, ratio, seed, offset, dbias=True)
    for row in rows_to_check(R, C).tolist():   # (a row starts at a multiple of 4)
        keep = tr.dropout_keep(C, ratio, seed, offset, first=row * C)
        xr, rr = (t[row].double().cpu().numpy() for t in (x, r))
        kept = np.where(keep, 2 * (xr + b.double().cpu().numpy()), 0.0)
        assert_within(y[row].cpu(), kept + rr, U32 * (3 * np.abs(kept) + np.abs(kept + rr)), "dropout")
        assert_within(dx[row].cpu(), np.where(keep, 2 * xr, 0.0), 3 * U32 * np.abs(2 * xr), "dropout dX")
    # (2 dY is exact, so dX holds the very terms of dbias)
    s = chunked(R, lambda a, e: torch.stack([dx[a:e].double().sum(0), dx[a:e].double().abs().sum(0)]), 1 << 14)
    assert_within(dbias.cpu(), s[0].cpu().numpy(), 64 * U32 * s[1].cpu().numpy(), "dropout dbias")
