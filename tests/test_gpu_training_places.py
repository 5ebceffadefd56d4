"""GroupNorm's gradient with dY, X and dX at offsets of their own within 16 bytes, in every
form, and the sums of the token gradient past 2^31 elements."""
import pytest
import torch

from gen import synth
from oracle import training as tr
from tests._helpers import U32, Guarded, offset_copy
from tests._training import assert_within, group_norm_inputs

pytestmark = pytest.mark.gpu

EPS = 1e-5
FORMS = [((1100, 1, 1024), 8), ((700, 1, 320), 4), ((9, 1, 4096), 2), ((3, 17, 64), 4), ((3, 17, 80), 8), ((3, 21, 189), 9),
         ((3, 1, 5001), 3), ((700, 1, 76), 4), ((320, 3, 27), 9), ((2, 3000, 64), 4), ((2, 1024, 320), 32), ((1, 300, 12288), 32),
         ((2, 5000, 27), 9), ((3, 1331, 189), 9), ((2, 400, 1530), 9)]


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("x_at,dy_at,dx_at", [(0, 8, 0), (4, 12, 4), (8, 0, 4), (0, 4, 4), (4, 4, 0)])
@pytest.mark.parametrize("shape,groups", FORMS)
def test_operands_at_their_own_offsets(lib, dtype, shape, groups, x_at, dy_at, dx_at):
    d = group_norm_inputs(shape, dtype, sum(shape) + x_at + dy_at)
    x, dy = offset_copy(d["X"], x_at)[1], offset_copy(d["dY"], dy_at)[1]
    gamma, beta = d["gamma"].cuda(), d["beta"].cuda()
    dx = Guarded(shape, x.dtype, offset_bytes=dx_at)
    _, mean, inv = lib.ep_group_norm(x, gamma, beta, groups, EPS, lib.EP_ACT_SILU, mean=True, inv_std_dev=True)
    _, dg, db = lib.ep_group_norm_grad(dy, x, gamma, beta, mean, inv, groups, lib.EP_ACT_SILU, dX=dx.tensor)
    torch.cuda.synchronize()
    dx.check()
    o = tr.group_norm_grad(d["dY"], d["X"], d["gamma"], d["beta"], mean.cpu(), inv.cpu(), groups, True)
    assert_within(dx.tensor.cpu(), o["dX"], 64 * U32 * o["dX_scale"], "gn dX")
    assert_within(dg.cpu(), o["dgamma"], 64 * U32 * o["dgamma_scale"], "gn dgamma")
    assert_within(db.cpu(), o["dbeta"], 64 * U32 * o["dbeta_scale"], "gn dbeta")


def test_token_gradient_sums_past_2_31_elements(lib):
    # dgamma = sum of dY h with h from the returned statistics: 64 half steps of the sum of the
    # terms' magnitudes, as everywhere
    C, groups = 4096, 32
    N = (1 << 31) // C + 77
    x = synth.device_normal((N, 1, C), "f16", seed=85)
    dy = synth.device_normal((N, 1, C), "f16", seed=86)
    gamma = synth.device_normal((C,), "f16", seed=87, std=0.2) + 1
    _, mean, inv = lib.ep_group_norm(x, gamma, None, groups, EPS, mean=True, inv_std_dev=True)
    dx, dgamma, dbeta = lib.ep_group_norm_grad(dy, x, gamma, None, mean, inv, groups)
    del dx
    sums = torch.zeros(4, C, dtype=torch.float64, device="cuda")
    step = 1 << 14
    for a in range(0, N, step):
        b = min(N, a + step)
        v, w = x[a:b].double().view(b - a, groups, -1), dy[a:b, 0].double()
        t = w * ((v - mean[a:b, :, None].double()) * inv[a:b, :, None].double()).view(b - a, C)
        sums += torch.stack([t.sum(0), t.abs().sum(0), w.sum(0), w.abs().sum(0)])
    dg, dg_abs, db, db_abs = (s.cpu().numpy() for s in sums)
    assert_within(dgamma.cpu(), dg, 64 * U32 * dg_abs, "gn dgamma")
    assert_within(dbeta.cpu(), db, 64 * U32 * db_abs, "gn dbeta")
    del x, dy
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
