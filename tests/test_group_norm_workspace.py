"""GroupNorm's scratch: of the order of the data for every number of groups.

A part (16 bytes, 8 in the gradient) belongs to a chunk and to a group that a tile
of the chunk meets: at most G + 2 tiles of them to a chunk, and a tile has 1024
channels or more, so with one group to a channel and one position to a chunk scratch
is 16 bytes (8) a value, and 8 a (sample, group) for the statistics.  The gradient
adds 8 bytes a channel for each row of blocks.
"""
import pytest
import torch

import transformer_epilogue_gb300 as te


@pytest.fixture(scope="module", autouse=True)
def built():
    from transformer_epilogue_gb300 import build
    build.build()


SHAPES = [((1, 64, 65536), 65536), ((1, 8, 1 << 20), 1 << 20), ((1, 1, 1 << 24), 1 << 24), ((1, 16, 1 << 20), 1 << 20),
          ((3, 5, 16384), 4096), ((40, 100, 16384), 4096), ((1, 64, 65536), 256), ((2, 1000, 12288), 32),
          ((1, 1000, 40000), 40000), ((16, 4, 131072), 1024)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_scratch_grows_with_the_groups(dtype, shape, groups):
    n, s, c = shape
    values, es = n * s * c, 4 if dtype == torch.float32 else 2
    vw = 16 // es
    rows = max(4, s // 304)   # positions of a chunk, where there are as many
    parts = -(-s // min(rows, s)) * n * (groups + 2 * (c // 1024 + 1))
    stats = 8 * n * groups + 32
    assert te.ep_group_norm_workspace_size(dtype, shape, groups) <= 16 * parts + stats
    # the channels' sums: a row for each CTA of a walk row's tiles, two an SM of 152 (at least one)
    sums = 8 * c * max(1, 304 // max(1, c // (256 * vw)))
    assert te.ep_group_norm_grad_workspace_size(dtype, shape, groups) <= 8 * parts + stats + sums
    assert te.ep_group_norm_workspace_size(dtype, shape, groups) <= 26 * values + (1 << 16)


@pytest.mark.parametrize("shape,groups", [((1, 64, 65536), 65536), ((1, 8, 1 << 20), 1 << 20)])
def test_scratch_of_channels_as_groups(shape, groups):
    # 8 positions or more to a channel: no more than a few times the data
    data = 2 * shape[0] * shape[1] * shape[2]
    for size in (te.ep_group_norm_workspace_size, te.ep_group_norm_grad_workspace_size):
        assert size(torch.float16, shape, groups) <= 3 * data
