"""GroupNorm, form by form: what must not depend on alignment, aliasing, scratch,
streams or other groups.  Each shape takes another kernel; results are compared
bit for bit with a plain call, which the shape tests compare with the oracle."""
import numpy as np
import pytest
import torch

from oracle import training as tr
from tests._helpers import U32, Guarded, offset_copy
from tests._training import assert_within, group_norm_inputs

pytestmark = pytest.mark.gpu

FORMS = [
    ((1100, 1, 1024), 8, "bf16"), ((1200, 1, 512), 4, "f32"),                       # many tokens
    ((9, 1, 320), 4, "f16"), ((5, 1, 8192), 8, "f16"), ((70, 1, 96), 3, "f32"),     # tokens
    ((3, 17, 64), 4, "f16"), ((3, 17, 80), 8, "f16"), ((3, 21, 189), 9, "f16"), ((3, 1, 5001), 3, "f16"),
    ((700, 1, 76), 4, "bf16"), ((320, 3, 27), 9, "f32"), ((300, 1, 2295), 9, "f32"),  # small samples
    ((2, 3000, 64), 4, "f16"), ((2, 4096, 320), 32, "f16"), ((1, 300, 12288), 32, "bf16"), ((40, 900, 32), 4, "f16"),
    ((2, 5000, 27), 9, "f16"), ((3, 1331, 189), 9, "f32"),                          # large samples
    ((2, 400, 1530), 9, "bf16"), ((30, 1, 9001), 1, "f16"),                         # the general kernels
]
EPS = 1e-5


def both(lib, t, groups, **kw):
    """Y, mean, inv, dX, dgamma, dbeta of t."""
    f = lib.ep_group_norm(t["X"], t["gamma"], t["beta"], groups, EPS, lib.EP_ACT_SILU, mean=True, inv_std_dev=True, **kw)
    return f + lib.ep_group_norm_grad(t["dY"], t["X"], t["gamma"], t["beta"], f[1], f[2], groups, lib.EP_ACT_SILU, **kw)


def case(shape, groups, dtype):
    d = group_norm_inputs(shape, dtype, sum(shape) + groups)
    return {k: v.cuda() for k, v in d.items()}


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("shape,groups,dtype", FORMS)
def test_parameters_and_statistics_anywhere(lib, shape, groups, dtype):
    t = case(shape, groups, dtype)
    want = both(lib, t, groups)
    es = t["X"].element_size()
    keep = [offset_copy(t[k], es) for k in ("gamma", "beta")]
    u = dict(t, gamma=keep[0][1], beta=keep[1][1])
    mean, inv = (Guarded((shape[0], groups), torch.float32, offset_bytes=4) for _ in range(2))
    dg, db = (Guarded((shape[-1],), t["X"].dtype, offset_bytes=es) for _ in range(2))
    y, _, _ = lib.ep_group_norm(u["X"], u["gamma"], u["beta"], groups, EPS, lib.EP_ACT_SILU, mean=mean.tensor,
                                inv_std_dev=inv.tensor)
    dx, _, _ = lib.ep_group_norm_grad(u["dY"], u["X"], u["gamma"], u["beta"], mean.tensor, inv.tensor, groups,
                                      lib.EP_ACT_SILU, dgamma=dg.tensor, dbeta=db.tensor)
    torch.cuda.synchronize()
    for g in (mean, inv, dg, db):
        g.check()
    assert same((y, mean.tensor, inv.tensor, dx, dg.tensor, db.tensor), want)


@pytest.mark.parametrize("shape,groups,dtype", FORMS)
def test_in_place(lib, shape, groups, dtype):
    t = case(shape, groups, dtype)
    want = both(lib, t, groups)
    x = t["X"].clone()
    lib.ep_group_norm(x, t["gamma"], t["beta"], groups, EPS, lib.EP_ACT_SILU, Y=x)
    assert torch.equal(x, want[0])
    for alias in ("dY", "X"):
        u = dict(t, **{alias: t[alias].clone()})
        got = lib.ep_group_norm_grad(u["dY"], u["X"], u["gamma"], u["beta"], want[1], want[2], groups, lib.EP_ACT_SILU,
                                     dX=u[alias])
        assert same(got, want[3:])


@pytest.mark.parametrize("shape,groups,dtype", FORMS)
def test_scratch_streams_and_graphs(lib, shape, groups, dtype):
    t = case(shape, groups, dtype)
    want = both(lib, t, groups)
    torch.cuda.synchronize()
    need = max(lib.ep_group_norm_workspace_size(t["X"].dtype, shape, groups),
               lib.ep_group_norm_grad_workspace_size(t["X"].dtype, shape, groups))
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN everywhere: contents do not matter
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(lib, t, groups, workspace=ws[:need], stream=s)
    torch.cuda.synchronize()
    assert same(got, want)
    # two graphs that share the scratch, replayed in turn
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both(lib, t, groups, workspace=ws[:need]))
        graphs.append(g)
    for o in outs[0] + outs[1]:
        o.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert same(outs[0], want) and same(outs[1], want)
    assert bool((ws[need:] == 0xFF).all()), "write behind the workspace"
    assert lib.ep_pipeline_timeouts() == 0


@pytest.mark.parametrize("shape,groups,dtype", FORMS)
def test_non_finite_values_stay_in_their_group(lib, shape, groups, dtype):
    t = case(shape, groups, dtype)
    want = both(lib, t, groups)
    n, c, s = shape[0], shape[-1], shape[1] // 2
    d = c // groups
    bad_n, bad_g = n // 2, groups // 2
    x = t["X"].clone()
    x[bad_n, s, bad_g * d + d // 2] = float("inf")
    got = both(lib, dict(t, X=x), groups)
    hit = torch.zeros((n, groups), dtype=torch.bool, device="cuda")
    hit[bad_n, bad_g] = True
    assert torch.equal(got[1][~hit], want[1][~hit]) and torch.equal(got[2][~hit], want[2][~hit])
    apart = ~hit.view(n, 1, groups, 1).expand(n, shape[1], groups, d).reshape(shape)
    assert torch.equal(got[0][apart], want[0][apart])
    assert torch.equal(got[3][apart], want[3][apart])
    assert bool(got[0][~apart].isnan().any())
    channels = torch.ones(c, dtype=torch.bool, device="cuda")
    channels[bad_g * d:(bad_g + 1) * d] = False
    assert torch.equal(got[4][channels], want[4][channels]) and torch.equal(got[5][channels], want[5][channels])


@pytest.mark.parametrize("shape,groups,dtype", FORMS)
def test_outliers_where_the_centre_is_taken(lib, shape, groups, dtype):
    # The kernels take their values relative to a centre, the median of three of
    # them (for a chunk or for the sample).  Two of the sample's three are made
    # outliers: the centre lies k standard deviations off the mean, and the sums of
    # squares about it, n (1 + k^2) sigma^2 with a relative error of at most 64 half
    # steps as in the plain case, give the variance (1 + k^2) times that error and
    # 1 / sqrt half of it; the sums n k sigma give the mean 16 k half steps of sigma.
    d = group_norm_inputs(shape, dtype, 5)
    g = d["X"].view(shape[0], shape[1], groups, -1)
    g[:, 0, :, 0] = 40.0
    g[:, shape[1] // 2, :, g.shape[-1] // 2] = 40.0
    o = tr.group_norm(d["X"], d["gamma"], d["beta"], groups, EPS)
    _, mean, inv = lib.ep_group_norm(d["X"].cuda(), d["gamma"].cuda(), d["beta"].cuda(), groups, EPS, mean=True,
                                     inv_std_dev=True)
    sigma = 1.0 / o["inv_std_dev"]
    k = np.abs(40.0 - o["mean"]) / sigma
    assert_within(mean.cpu(), o["mean"], 16 * U32 * (np.abs(o["mean"]) + sigma * (1 + k) + 40.0), "gn mean")
    assert_within(inv.cpu(), o["inv_std_dev"], 64 * U32 * o["inv_std_dev"] * (1 + k * k), "gn inv")
