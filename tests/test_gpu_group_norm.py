"""GroupNorm and its gradient (through the C ABI) against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import training as tr
from tests._helpers import U32, Guarded, assert_bit_exact, offset_copy, to_np64
from tests._training import assert_within, group_norm_inputs, norm_delta

pytestmark = pytest.mark.gpu

# (shape (N, positions..., C), groups)
SHAPES = [
    ((1, 1, 8), 1), ((1, 1, 1), 1), ((2, 1, 3), 3),       # one token; groups of one value
    ((5, 1, 256), 8), ((37, 1, 96), 4), ((700, 1, 64), 2),  # tokens
    ((300, 2, 15), 3), ((1300, 1, 24), 3), ((1500, 1, 9), 3),
    ((2, 7, 10), 2), ((3, 33, 189), 9), ((2, 5, 7, 30), 6),  # rows that are no multiple of 16 bytes
    ((2, 64, 320), 32), ((1, 257, 640), 32), ((2, 100, 128), 128), ((2, 50, 128), 1),
    ((1, 9, 4104), 27), ((2, 3, 2055), 5), ((1, 4, 8192), 64),   # rows wider than a block of threads
    ((1, 5000, 32), 8), ((2, 3000, 1), 1), ((1, 2777, 5), 5), ((1, 700, 3), 1),  # few channels
    ((2, 9973, 40), 4),
    ((2, 1024, 320), 32), ((1, 2048, 96), 96), ((3, 1331, 189), 9), ((1, 4096, 64), 2),  # more than a block holds
    ((4503, 1, 1024), 8), ((1103, 1, 4352), 17), ((9001, 1, 544), 17),  # many tokens
    # tokens whose groups are 10, 5, 128, 256 and 18 fragments (fp16)
    ((700, 1, 320), 4), ((3, 1, 1280), 32), ((300, 1, 8192), 8), ((41, 1, 4096), 2), ((5, 1, 432), 3),
    ((1000, 1, 768), 3), ((1, 1, 544), 1),
    # many small samples, several to a block or one block after another, that start anywhere
    ((700, 1, 76), 4), ((650, 3, 27), 9), ((400, 2, 675), 3), ((1100, 5, 117), 9), ((333, 1, 744), 8),
    ((900, 1, 2976), 32), ((310, 8, 4), 4), ((500, 2, 384), 64), ((2000, 2, 1), 1), ((160, 1, 4095), 5),
    ((77, 9, 1044), 9), ((40, 1, 5001), 3), ((400, 1, 1827), 9), ((200, 2, 3999), 3), ((300, 1, 2295), 9), ((500, 1, 8160), 32), ((180, 1, 7999), 1), ((3, 2, 5001), 1), ((2, 401, 1530), 9), ((1, 2500, 1044), 9), ((3, 700, 747), 9),
    ((1, 70000, 64), 4), ((2, 30011, 33), 3), ((1, 300, 12288), 32),  # large samples
]


def stats_close(mean, inv, o, std):
    assert_within(mean, o["mean"], 16 * U32 * (np.abs(o["mean"]) + std), "gn mean")
    assert_within(inv, o["inv_std_dev"], 64 * U32 * o["inv_std_dev"], "gn inv")


def forward(lib, d, groups, eps, silu, offset=0, in_place=False):
    x = offset_copy(d["X"], offset)[1] if offset else d["X"].cuda()
    n = d["X"].shape[0]
    y = Guarded(d["X"].shape, d["X"].dtype, offset_bytes=offset)
    mean, inv = Guarded((n, groups), torch.float32), Guarded((n, groups), torch.float32)
    if in_place:
        y.tensor.copy_(x)
        x = y.tensor
    lib.ep_group_norm(x, d["gamma"].cuda(), None if d["beta"] is None else d["beta"].cuda(), groups, eps,
                      lib.EP_ACT_SILU if silu else lib.EP_ACT_NONE, Y=y.tensor, mean=mean.tensor,
                      inv_std_dev=inv.tensor)
    torch.cuda.synchronize()
    for g in (y, mean, inv):
        g.check()
    return y.tensor.cpu(), mean.tensor.cpu(), inv.tensor.cpu()


def check_forward(lib, d, groups, eps, silu, std=1.0, **kw):
    y, mean, inv = forward(lib, d, groups, eps, silu, **kw)
    o = tr.group_norm(d["X"], d["gamma"], d["beta"], groups, eps, silu)
    stats_close(mean, inv, o, std)
    delta = norm_delta(o["mean"], o["inv_std_dev"], d["gamma"], groups, d["X"].shape[-1])
    n, c = d["X"].shape[0], d["X"].shape[-1]
    assert_within(y, o["Y"].reshape(n, -1, c), delta, "gn")
    return y


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_group_norm_shapes(lib, dtype, shape, groups):
    seed = sum(shape) + groups
    d = group_norm_inputs(shape, dtype, seed, beta=seed % 3 != 0)
    check_forward(lib, d, groups, 1e-5, silu=seed % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape,groups", [((2, 33, 64), 4), ((3, 21, 189), 9), ((6, 1, 96), 4)])
@pytest.mark.parametrize("offset", [4, 8, 12])
def test_group_norm_alignment(lib, dtype, shape, groups, offset):
    d = group_norm_inputs(shape, dtype, 11 + offset)
    check_forward(lib, d, groups, 1e-5, True, offset=offset)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_group_norm_shapes_apart(lib, dtype, shape, groups):
    # an output at another offset than the input: the split form, for every shape
    d = group_norm_inputs(shape, dtype, 17 + sum(shape))
    x, dy, gamma, beta = (d[k].cuda() for k in ("X", "dY", "gamma", "beta"))
    es = x.element_size()
    y, dx = (Guarded(shape, x.dtype, offset_bytes=es) for _ in range(2))
    _, mean, inv = lib.ep_group_norm(x, gamma, beta, groups, 1e-5, lib.EP_ACT_SILU, Y=y.tensor, mean=True,
                                     inv_std_dev=True)
    _, dg, db = lib.ep_group_norm_grad(dy, x, gamma, beta, mean, inv, groups, lib.EP_ACT_SILU, dX=dx.tensor)
    torch.cuda.synchronize()
    y.check()
    dx.check()
    n, c = shape[0], shape[-1]
    o = tr.group_norm(d["X"], d["gamma"], d["beta"], groups, 1e-5, True)
    stats_close(mean.cpu(), inv.cpu(), o, 1.0)
    assert_within(y.tensor.cpu(), o["Y"].reshape(n, -1, c),
                  norm_delta(o["mean"], o["inv_std_dev"], d["gamma"], groups, c), "gn")
    o = tr.group_norm_grad(d["dY"], d["X"], d["gamma"], d["beta"], mean.cpu(), inv.cpu(), groups, True)
    assert_within(dx.tensor.cpu(), o["dX"], 64 * U32 * o["dX_scale"], "gn dX")
    assert_within(dg.cpu(), o["dgamma"], 64 * U32 * o["dgamma_scale"], "gn dgamma")
    assert_within(db.cpu(), o["dbeta"], 64 * U32 * o["dbeta_scale"], "gn dbeta")


def test_group_norm_different_alignments(lib):
    d = group_norm_inputs((3, 21, 40), "f16", 5)
    x = offset_copy(d["X"], 2)[1]
    y = Guarded(d["X"].shape, torch.float16, offset_bytes=8)
    lib.ep_group_norm(x, d["gamma"].cuda(), d["beta"].cuda(), 4, Y=y.tensor)
    torch.cuda.synchronize()
    y.check()
    o = tr.group_norm(d["X"], d["gamma"], d["beta"], 4, 1e-5)
    assert_within(y.tensor.cpu(), o["Y"], norm_delta(o["mean"], o["inv_std_dev"], d["gamma"], 4, 40), "gn")


@pytest.mark.parametrize("shape,groups", [((2, 33, 64), 4), ((3, 21, 189), 9), ((6, 1, 96), 4), ((1, 900, 512), 32)])
def test_group_norm_in_place(lib, shape, groups):
    d = group_norm_inputs(shape, "bf16", 21)
    a = check_forward(lib, d, groups, 1e-5, True)
    b = check_forward(lib, d, groups, 1e-5, True, in_place=True)
    assert_bit_exact(a, b)


@pytest.mark.parametrize("mean,std", [(1000.0, 1.0), (-3e4, 0.5), (0.0, 1e-3), (1e-3, 1e6)])
def test_group_norm_large_mean_keeps_the_variance(lib, mean, std):
    # float32: E[x^2] - mu^2 would lose the variance here
    d = group_norm_inputs((2, 700, 48), "f32", 31, mean=mean, std=std)
    check_forward(lib, d, 6, 1e-12, False, std=std)


def test_group_norm_constant_groups(lib):
    # variance 0: h = 0, so y = beta (SiLU of it), whatever epsilon > 0
    d = group_norm_inputs((2, 50, 24), "f32", 41)
    d["X"] = torch.full_like(d["X"], 3.25)
    y, mean, inv = forward(lib, d, 4, 1e-5, False)
    assert torch.equal(y, d["beta"].expand_as(y))
    assert torch.equal(mean, torch.full_like(mean, 3.25))


def test_group_norm_non_finite_values_stay_in_their_group(lib):
    d = group_norm_inputs((3, 40, 32), "f16", 51)
    x = d["X"].clone()
    x[1, 7, 9] = float("nan")     # group 2 of 8 (channels 8..11)
    x[2, 3, 30] = float("inf")    # group 7
    clean, _, _ = forward(lib, d, 8, 1e-5, True)
    y, mean, inv = forward(lib, dict(d, X=x), 8, 1e-5, True)
    assert torch.isnan(y[1, :, 8:12]).all() and torch.isnan(y[2, :, 28:32]).any()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1, :, 8:12] = False
    keep[2, :, 28:32] = False
    assert torch.equal(y[keep], clean[keep])


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------

def gradient(lib, d, groups, silu, mean, inv, offset=0, alias=None):
    c = d["X"].shape[-1]
    place = (lambda t: offset_copy(t, offset)[1]) if offset else (lambda t: t.cuda())
    x, dy = place(d["X"]), place(d["dY"])
    dx = Guarded(d["X"].shape, d["X"].dtype, offset_bytes=offset)
    if alias == "dY":
        dx.tensor.copy_(dy)
        dy = dx.tensor
    elif alias == "X":
        dx.tensor.copy_(x)
        x = dx.tensor
    dg, db = Guarded((c,), d["X"].dtype), Guarded((c,), d["X"].dtype)
    lib.ep_group_norm_grad(dy, x, d["gamma"].cuda(), None if d["beta"] is None else d["beta"].cuda(), mean.cuda(),
                           inv.cuda(), groups, lib.EP_ACT_SILU if silu else lib.EP_ACT_NONE, dX=dx.tensor,
                           dgamma=dg.tensor, dbeta=db.tensor)
    torch.cuda.synchronize()
    for g in (dx, dg, db):
        g.check()
    return dx.tensor.cpu(), dg.tensor.cpu(), db.tensor.cpu()


def saved_stats(d, groups, eps=1e-5):
    f = tr.group_norm(d["X"], d["gamma"], d["beta"], groups, eps)
    return torch.from_numpy(f["mean"]).float(), torch.from_numpy(f["inv_std_dev"]).float()


def check_gradient(lib, d, groups, silu, **kw):
    mean, inv = saved_stats(d, groups)
    dx, dg, db = gradient(lib, d, groups, silu, mean, inv, **kw)
    o = tr.group_norm_grad(d["dY"], d["X"], d["gamma"], d["beta"], mean, inv, groups, silu)
    assert_within(dx, o["dX"], 64 * U32 * o["dX_scale"], "gn dX")
    assert_within(dg, o["dgamma"], 64 * U32 * o["dgamma_scale"], "gn dgamma")
    assert_within(db, o["dbeta"], 64 * U32 * o["dbeta_scale"], "gn dbeta")
    return dx, dg, db


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_group_norm_grad_shapes(lib, dtype, shape, groups):
    seed = sum(shape) + groups
    d = group_norm_inputs(shape, dtype, seed, beta=seed % 3 != 0)
    check_gradient(lib, d, groups, silu=seed % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape,groups", [((2, 33, 64), 4), ((3, 21, 189), 9), ((6, 1, 96), 4)])
@pytest.mark.parametrize("offset", [4, 8, 12])
def test_group_norm_grad_alignment(lib, dtype, shape, groups, offset):
    d = group_norm_inputs(shape, dtype, 13 + offset)
    check_gradient(lib, d, groups, True, offset=offset)


@pytest.mark.parametrize("alias", ["dY", "X"])
@pytest.mark.parametrize("shape,groups", [((2, 33, 64), 4), ((3, 21, 189), 9), ((6, 1, 96), 4), ((1, 900, 512), 32)])
def test_group_norm_grad_in_place(lib, alias, shape, groups):
    d = group_norm_inputs(shape, "f16", 23)
    a = check_gradient(lib, d, groups, True)
    b = check_gradient(lib, d, groups, True, alias=alias)
    for p, q in zip(a, b):
        assert_bit_exact(p, q)


def test_group_norm_grad_without_parameter_gradients(lib):
    d = group_norm_inputs((2, 33, 64), "f32", 61)
    mean, inv = saved_stats(d, 4)
    full = gradient(lib, d, 4, True, mean, inv)
    args = (d["dY"].cuda(), d["X"].cuda(), d["gamma"].cuda(), d["beta"].cuda(), mean.cuda(), inv.cuda(), 4,
            lib.EP_ACT_SILU)
    dx, dg, db = lib.ep_group_norm_grad(*args, dgamma=None, dbeta=None)
    assert dg is None and db is None and torch.equal(dx.cpu(), full[0])
    dx, dg, db = lib.ep_group_norm_grad(*args, dgamma=None)
    assert dg is None and torch.equal(db.cpu(), full[2])
    dx, dg, db = lib.ep_group_norm_grad(*args, dbeta=None)
    assert db is None and torch.equal(dg.cpu(), full[1])


def test_group_norm_grad_against_differences(lib):
    # the kernels' own forward pass, in float32, at x + step and x - step along
    # random directions: d/dt sum(w * y(x + t v)) = sum(dX * v)
    d = group_norm_inputs((2, 40, 24), "f32", 71)
    x, g, b, w = (d[k].cuda() for k in ("X", "gamma", "beta", "dY"))
    _, mean, inv = lib.ep_group_norm(x, g, b, 4, 1e-5, lib.EP_ACT_SILU, mean=True, inv_std_dev=True)
    dx, dg, db = lib.ep_group_norm_grad(w, x, g, b, mean, inv, 4, lib.EP_ACT_SILU)
    gen = torch.Generator().manual_seed(72)
    step = 2.0 ** -7

    def value(x, g, b):
        y, _, _ = lib.ep_group_norm(x, g, b, 4, 1e-5, lib.EP_ACT_SILU)
        return float((y.double() * w.double()).sum())

    # central differences: the values are float32 y (off by about 1e-6 of |y| <
    # 6, 1920 of them with random signs: 3e-4), over 2 step = 2^-6: 0.02; the
    # third derivative's share is step^2 / 6 of O(100): 0.001
    tol = 0.03
    for k in range(3):
        vx, vg, vb = (torch.randn(t.shape, generator=gen).cuda() for t in (x, g, b))
        want = float((dx.double() * vx).sum() + (dg.double() * vg).sum() + (db.double() * vb).sum())
        scale = float(torch.sqrt((vx * vx).sum() + (vg * vg).sum() + (vb * vb).sum()))
        vx, vg, vb = vx / scale, vg / scale, vb / scale
        got = (value(x + step * vx, g + step * vg, b + step * vb)
               - value(x - step * vx, g - step * vg, b - step * vb)) / (2 * step)
        assert abs(got - want / scale) < tol


def test_group_norm_repeats_bit_for_bit(lib):
    d = group_norm_inputs((3, 2000, 96), "bf16", 81)
    t = {k: d[k].cuda() for k in d}
    first = None
    for _ in range(4):
        y, mean, inv = lib.ep_group_norm(t["X"], t["gamma"], t["beta"], 8, mean=True, inv_std_dev=True)
        out = (y, mean, inv) + lib.ep_group_norm_grad(t["dY"], t["X"], t["gamma"], t["beta"], mean, inv, 8)
        if first is None:
            first = [o.clone() for o in out]
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_group_norm_empty_tensors(lib):
    for shape in ((0, 4, 8), (3, 0, 8)):
        x = torch.empty(shape, dtype=torch.float16, device="cuda")
        g = torch.ones(8, dtype=torch.float16, device="cuda")
        y, mean, inv = lib.ep_group_norm(x, g, g, 2, mean=True, inv_std_dev=True)
        assert y.shape == x.shape
        dx, dg, db = lib.ep_group_norm_grad(x, x, g, g, mean, inv, 2)
        assert dx.shape == x.shape and not dg.any() and not db.any()


def test_group_norm_own_stream_and_workspace(lib):
    d = group_norm_inputs((2, 3000, 64), "f16", 91)
    t = {k: d[k].cuda() for k in d}
    want = lib.ep_group_norm(t["X"], t["gamma"], t["beta"], 4, mean=True, inv_std_dev=True)
    need = lib.ep_group_norm_workspace_size(torch.float16, (2, 3000, 64), 4)
    ws = torch.full((need + 32,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN everywhere: contents do not matter
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = lib.ep_group_norm(t["X"], t["gamma"], t["beta"], 4, mean=True, inv_std_dev=True, workspace=ws[:need],
                            stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert bool((ws[need:] == 0xFF).all())
    if need:
        with pytest.raises(lib.EpError) as e:
            lib.ep_group_norm(t["X"], t["gamma"], t["beta"], 4, workspace=ws[:need - 16])
        assert e.value.status == lib.EP_ERR_WORKSPACE


def test_group_norm_statistics_match_skip_layer_norm(lib):
    # one group over one position is the layer norm of the row
    d = group_norm_inputs((64, 1, 768), "f32", 95)
    x, g, b = d["X"].cuda(), d["gamma"].cuda(), d["beta"].cuda()
    y, mean, inv = lib.ep_group_norm(x, g, b, 1, 1e-5, mean=True, inv_std_dev=True)
    ln, _, m2, i2 = lib.ep_skip_layer_norm_ex(x, torch.zeros_like(x), g, b, epsilon=1e-5, mean=True,
                                              inv_std_dev=True)
    o = tr.group_norm(d["X"], d["gamma"], d["beta"], 1, 1e-5)
    assert_within(ln.cpu(), to_np64(y), 2e-5, "gn against layer norm")
    stats_close(mean.cpu(), inv.cpu(), o, 1.0)
    stats_close(m2.cpu().view(64, 1), i2.cpu().view(64, 1), o, 1.0)
