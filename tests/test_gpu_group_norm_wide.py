"""GroupNorm of wide rows in many groups (walk rows of many tiles, each of which meets
a part of the groups), aligned and not, against the definition in float64.

Tolerances: those of the shape tests (tests/_training.py): the same arithmetic.
"""
import pytest
import torch

from oracle import training as tr
from tests._helpers import U32, Guarded, offset_copy
from tests._training import assert_within, group_norm_inputs, norm_delta

pytestmark = pytest.mark.gpu

EPS = 1e-5
# groups inside a tile, groups over two tiles and over many, groups of one channel, rows that are
# no multiple of 16 bytes, a tile that ends inside a group
SHAPES = [((1, 64, 65536), 65536, "f16"), ((1, 6, 40000), 10000, "f16"), ((2, 3, 24576), 24, "bf16"), ((3, 9, 8200), 1025, "f32"),
          ((2, 40, 12288), 3, "f16"), ((1, 5, 40001), 40001, "f16"), ((2, 3, 30003), 10001, "bf16"), ((1, 7, 21021), 3003, "f32"),
          ((2, 2, 9009), 1001, "f16"), ((40, 1, 20000), 2500, "f16"), ((5, 1, 33333), 11111, "f32"), ((1, 1, 1 << 20), 1 << 18, "f16"),
          ((300, 2, 8224), 257, "bf16"), ((2, 70, 4112), 4112, "f16"), ((1, 300, 16400), 2050, "f16")]


@pytest.mark.parametrize("shape,groups,dtype", SHAPES)
@pytest.mark.parametrize("place", ["aligned", "offset", "results apart", "dY apart"])
def test_wide_rows(lib, shape, groups, dtype, place):
    d = group_norm_inputs(shape, dtype, sum(shape) % 1000 + groups)
    n, c = shape[0], shape[-1]
    es = d["X"].element_size()
    x_at, dy_at, y_at = {"aligned": (0, 0, 0), "offset": (es, es, es), "results apart": (0, 0, es),
                         "dY apart": (es, 16 - es, 0)}[place]
    x, dy = offset_copy(d["X"], x_at)[1], offset_copy(d["dY"], dy_at)[1]
    gamma, beta = d["gamma"].cuda(), d["beta"].cuda()
    y, dx = (Guarded(shape, x.dtype, offset_bytes=y_at) for _ in range(2))
    need = (lib.ep_group_norm_workspace_size(x.dtype, shape, groups),
            lib.ep_group_norm_grad_workspace_size(x.dtype, shape, groups))
    ws = torch.full((max(need) + 256,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN everywhere
    _, mean, inv = lib.ep_group_norm(x, gamma, beta, groups, EPS, lib.EP_ACT_SILU, Y=y.tensor, mean=True,
                                     inv_std_dev=True, workspace=ws[:need[0]])
    ws.fill_(0xFF)
    _, dg, db = lib.ep_group_norm_grad(dy, x, gamma, beta, mean, inv, groups, lib.EP_ACT_SILU, dX=dx.tensor,
                                       workspace=ws[:need[1]])
    torch.cuda.synchronize()
    y.check()
    dx.check()
    assert bool((ws[need[1]:] == 0xFF).all()), "write behind the workspace"
    o = tr.group_norm(d["X"], d["gamma"], d["beta"], groups, EPS, True)
    # var + eps of a group of few values can be near eps, where 1/sqrt is that much steeper; the
    # variance's own error is 64 u of the squares' mean
    assert_within(mean.cpu(), o["mean"], 16 * U32 * (abs(o["mean"]) + 1.0), "gn mean")
    assert_within(inv.cpu(), o["inv_std_dev"], 64 * U32 * o["inv_std_dev"], "gn inv")
    # a group's values are up to |h| |mu| r u off in h: the mean's share, as in the shape tests
    assert_within(y.tensor.cpu(), o["Y"].reshape(n, -1, c),
                  norm_delta(o["mean"], o["inv_std_dev"], d["gamma"], groups, c), "gn")
    o = tr.group_norm_grad(d["dY"], d["X"], d["gamma"], d["beta"], mean.cpu(), inv.cpu(), groups, True)
    assert_within(dx.tensor.cpu(), o["dX"], 64 * U32 * o["dX_scale"], "gn dX")
    assert_within(dg.cpu(), o["dgamma"], 64 * U32 * o["dgamma_scale"], "gn dgamma")
    assert_within(db.cpu(), o["dbeta"], 64 * U32 * o["dbeta_scale"], "gn dbeta")
