"""GroupNorm's mean where it is much smaller than the values: it must not be rounded at
their size.

Values are multiples of 2^-12 below 2, so that sums about 0 of these groups are exact
in float32 (below 2^24 of those steps).  What is left is the rounding of 1 / n, of its
product with the sum, and a sum with 0: 3 half steps of the mean.  The places that a
centre may be taken from hold 1.5, 1.5 and -1.5.

Samples that take the split form are joined from the means of chunks, four positions or
more, each of which is rounded at its own size (3 half steps), as is its distance from the
one that the others are relative to: 4 half steps of the largest such mean besides.
The kernels for any C keep a mean for each channel, relative to a value of it: 4 half
steps of the values' size, 2.
"""
import pytest
import torch

from tests._helpers import U32

pytestmark = pytest.mark.gpu


def group(n, places, seed):
    """n values on the grid with a mean of about 2^-9, 1.5, 1.5 and -1.5 at the places."""
    g = torch.Generator().manual_seed(seed)
    k = torch.randint(-6000, 6001, (n,), generator=g)
    k[list(places)] = torch.tensor([6144, 6144, -6144])
    free = torch.ones(n, dtype=torch.bool)
    free[list(places)] = False
    rest = 8 * n - int(k.sum())
    each = rest // int(free.sum())
    k[free] += each
    k[free.nonzero()[:, 0][: rest - each * int(free.sum())]] += 1
    assert int(k.abs().max()) < 8192 * 4
    return k.double() / 4096


# (S, D): small samples of whole, odd and many channels a group; tokens
@pytest.mark.parametrize("s,d,token", [(3, 3, False), (5, 20, False), (7, 63, False), (40, 100, False), (50, 100, False),
                                       (11, 111, False), (11, 333, False), (1, 24, True), (1, 200, True), (1, 1000, True)])
@pytest.mark.parametrize("groups", [1, 3])
def test_mean_keeps_its_digits(lib, s, d, token, groups):
    n, form = s * d, {(50, 100, 3): "split", (11, 333, 1): "any C", (11, 333, 3): "any C"}.get((s, d, groups), "one pass")
    places = (0, 1, 3) if token else (0, s // 2 * d + d // 2, n - 1)
    x = torch.stack([group(n, places, 10 * n + k).view(s, d) for k in range(groups)], 1).reshape(1, s, groups * d)
    xs = x.float().cuda()
    assert torch.equal(xs.double().cpu(), x)
    gamma = torch.ones(groups * d, device="cuda")
    _, mean, _ = lib.ep_group_norm(xs, gamma, None, groups, mean=True, inv_std_dev=True)
    want = x.view(s, groups, d).mean((0, 2))
    size = {"one pass": 0.0, "any C": 2.0}.get(form)
    if size is None:
        size = float(x.view(s, groups, d).mean(2).unfold(0, 4, 1).mean(2).abs().max())
    assert bool(((mean[0].cpu().double() - want).abs() <= U32 * (3 * want.abs() + 4 * size)).all())
