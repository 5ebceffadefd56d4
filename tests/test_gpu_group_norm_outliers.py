"""GroupNorm's statistics where the values that a kernel might centre its sums on
are outliers: the variance must keep its digits all the same.

Ordinary values are +-(0.75 .. 1.25).  An outlying centre is told from the sums
(far off the mean in standard deviations) and replaced, so what is left is a
centre among the ordinary values or at the mean: at most 1.25 + |mean| off, k^2 <
2.5 variances.  A sum of squares about it is (1 + k^2) times the variance's, its
terms positive, so with sums of depth d the variance is off by (1 + k^2) (d + 8) u
at most, relatively, and 1/sqrt by half of that.  The mean is off by (d + 8) u
times the mean distance from the centre, and by two roundings of its own.

Depth: a thread adds 256 rows one after another, then come those sums and the
block's, at most 8 + 16 here; a fused block's threads add 8 rows, and a lane up to 128
columns; a token's lanes 8 values and 5 steps.
"""
import pytest
import torch

from tests._helpers import U32

pytestmark = pytest.mark.gpu

EPS = 1e-5
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def ordinary(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    size = torch.rand(shape, device="cuda", generator=g).mul_(0.5).add_(0.75)
    sign = torch.randint(0, 2, shape, device="cuda", generator=g, dtype=torch.int8).mul_(2).sub_(1)
    return size.mul_(sign).to(DT[dtype])


def definition(x, groups):
    """mean, 1/sqrt(var + eps) and the mean distance from the mean, in float64, (N, groups)."""
    mean, inv, dist = [], [], []
    for s in x:
        v = s.double().view(s.shape[0], groups, -1)
        m = v.mean((0, 2), keepdim=True)
        mean.append(m.flatten())
        inv.append(1.0 / torch.sqrt(((v - m) ** 2).mean((0, 2)) + EPS))
        dist.append((v - m).abs().mean((0, 2)))
    return torch.stack(mean), torch.stack(inv), torch.stack(dist)


def check(lib, x, groups, depth):
    c = x.shape[-1]
    gamma, beta = torch.ones(c, dtype=x.dtype, device="cuda"), torch.zeros(c, dtype=x.dtype, device="cuda")
    y, mean, inv = lib.ep_group_norm(x, gamma, beta, groups, EPS, mean=True, inv_std_dev=True)
    m, r, dist = definition(x, groups)
    off_mean = ((mean.double() - m).abs() / (U32 * ((depth + 8) * (dist + 1.5) + 2 * m.abs()))).max()
    off_inv = ((inv.double() - r).abs() / (U32 * 1.75 * (depth + 8) * r)).max()
    assert float(off_mean) <= 1 and float(off_inv) <= 1, (float(off_mean), float(off_inv))
    return y, mean, inv


# (N, S, C), groups, dtype.  So many samples that a chunk has many rows: one position a walk
# row, two tiles of one, whole samples that start anywhere, and the kernels for any C.
SPLIT = [((160, 1024, 516), 4, "f32"), ((160, 1024, 1032), 3, "f16"), ((160, 600, 2052), 9, "f32"),
         ((310, 2048, 255), 5, "f32"), ((310, 2048, 255), 1, "bf16"), ((210, 1024, 513), 9, "f32"), ((2, 3000, 64), 4, "f32")]


@pytest.mark.parametrize("shape,groups,dtype", SPLIT)
@pytest.mark.parametrize("where", ["first", "first and last", "middle and last"])
def test_outlying_positions(lib, shape, groups, dtype, where):
    x = ordinary(shape, dtype, sum(shape))
    s = shape[1]
    for name, at in (("first", 0), ("middle", s // 2), ("last", s - 1)):
        if name in where:
            x[:, at] = 300.0
    check(lib, x, groups, 256 + 24)


@pytest.mark.parametrize("shape,groups,dtype", SPLIT)
def test_outlying_first_value(lib, shape, groups, dtype):
    x = ordinary(shape, dtype, 1 + sum(shape))
    x.view(shape[0], shape[1], groups, -1)[:, 0, :, 0] = 30000.0
    check(lib, x, groups, 256 + 24)


@pytest.mark.parametrize("shape,groups,dtype", [((2, 3000, 64), 4, "f32"), ((2, 4096, 320), 32, "f16"),
                                                ((3, 1331, 189), 9, "f32"), ((1, 9000, 40), 1, "f32")])
def test_outlying_chunks(lib, shape, groups, dtype):
    # whole chunks (a share of the positions at both ends) away from the others
    x = ordinary(shape, dtype, 2 + sum(shape))
    s = shape[1]
    for a, b in ((0, s // 60), (s - s // 60, s)):
        x[:, a:b] += 300.0
    check(lib, x, groups, 256 + 24)


@pytest.mark.parametrize("shape,groups,dtype", [
    ((4, 16, 1024), 1, "f32"), ((4, 32, 1024), 1, "f16"), ((40, 16, 1000), 1, "f32"), ((4, 16, 1020), 3, "f32"),
    ((4, 30, 1007), 1, "f16"), ((500, 3, 333), 1, "f32"), ((500, 1, 2295), 1, "f32"), ((3, 40, 189), 9, "bf16")])
def test_outliers_in_a_small_sample(lib, shape, groups, dtype):
    x = ordinary(shape, dtype, 3 + sum(shape))
    g = x.view(shape[0], shape[1], groups, -1)
    for s, d in ((0, 0), (shape[1] // 2, g.shape[-1] // 2)):
        g[::2, s, :, d] = 1000.0   # (every second sample: the others' results must not depend on it)
    y, mean, inv = check(lib, x, groups, 8 + 8 + 128 + 16)
    clean = ordinary(shape, dtype, 3 + sum(shape))
    y0, mean0, inv0 = check(lib, clean, groups, 8 + 8 + 128 + 16)
    for a, b in ((y, y0), (mean, mean0), (inv, inv0)):
        assert torch.equal(a[1::2], b[1::2])


@pytest.mark.parametrize("shape,groups,dtype", [((2100, 1, 128), 1, "f32"), ((2100, 1, 256), 1, "bf16"),
                                                ((1500, 1, 1024), 4, "f16"), ((9, 1, 4096), 2, "f16")])
def test_outliers_in_a_token(lib, shape, groups, dtype):
    x = ordinary(shape, dtype, 4 + sum(shape))
    vw = 4 if dtype == "f32" else 8
    g = x.view(shape[0], shape[1], groups, -1)
    d = g.shape[-1]
    g[::2, :, :, 0] = 1000.0
    g[::2, :, :, d // 2 + vw // 2] = 1000.0
    y, mean, inv = check(lib, x, groups, 8 * max(1, d // 256) + 5)
    clean = ordinary(shape, dtype, 4 + sum(shape))
    y0, mean0, inv0 = check(lib, clean, groups, 8 * max(1, d // 256) + 5)
    for a, b in ((y, y0), (mean, mean0), (inv, inv0)):
        assert torch.equal(a[1::2], b[1::2])


@pytest.mark.parametrize("shape,groups,dtype", [((210, 40, 4098), 2, "f32"), ((210, 40, 4098), 3, "f32"), ((3, 700, 6006), 6, "f16"),
                                                ((40, 90, 12288), 4, "f32")])
def test_outlying_first_value_where_the_first_tile_lacks_the_group(lib, shape, groups, dtype):
    # (the parts of the walk row's first tile are empty for the later groups)
    x = ordinary(shape, dtype, 5 + sum(shape))
    x.view(shape[0], shape[1], groups, -1)[:, 0, :, 0] = 30000.0
    check(lib, x, groups, 256 + 24)


@pytest.mark.parametrize("shape,groups,dtype", [((160, 600, 516), 4, "f32"), ((310, 1200, 255), 5, "bf16"), ((210, 300, 513), 9, "f32"),
                                                ((40, 16, 1000), 1, "f16"), ((2100, 1, 256), 1, "bf16"), ((9, 1, 4096), 2, "f16")])
def test_second_sums_in_place_and_from_a_graph(lib, shape, groups, dtype):
    # what goes over its values again must not find its own results there
    x = ordinary(shape, dtype, 6 + sum(shape))
    for s in {0, shape[1] // 2, shape[1] - 1}:
        x[:, s].view(shape[0], groups, -1)[:, :, ::max(1, x.shape[-1] // groups // 2)] = 1000.0
    gamma, beta = torch.ones_like(x[0, 0]), torch.zeros_like(x[0, 0])
    want = lib.ep_group_norm(x, gamma, beta, groups, EPS, lib.EP_ACT_SILU, mean=True, inv_std_dev=True)
    own = x.clone()
    got = lib.ep_group_norm(own, gamma, beta, groups, EPS, lib.EP_ACT_SILU, Y=own, mean=True, inv_std_dev=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = lib.ep_group_norm(x, gamma, beta, groups, EPS, lib.EP_ACT_SILU, mean=True, inv_std_dev=True)
    for t in got:
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert lib.ep_pipeline_timeouts() == 0
