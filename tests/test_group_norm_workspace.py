"""GroupNorm's scratch: of the order of the data for every number of groups.

A part (16 bytes, 8 in the gradient) belongs to a chunk and to a group that a tile
of the chunk meets: at most G + 2 tiles of them to a chunk, and a tile has 1024
channels or more, so with one group to a channel and one position to a chunk scratch
is 16 bytes (8) a value, and 8 a (sample, group) for the statistics.  The gradient
adds 8 bytes a channel for each row of blocks.
"""
import json
import os
import subprocess
import sys

import pytest
import torch

import transformer_epilogue_gb300 as te

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


# taken by one launch without scratch where X and Y are aligned: tokens, small samples
ONE_LAUNCH = [((8, 1, 4096), 32), ((16384, 1, 8192), 64), ((8192, 1, 8192), 1024), ((300, 48, 256), 32), ((1, 40, 320), 32),
              ((700, 1, 76), 4), ((3, 21, 189), 9), ((1, 1, 1), 1)]
SPLIT = [((2, 4096, 320), 32), ((1, 64, 65536), 256), ((3, 1331, 189), 9), ((1, 1 << 17, 256), 2)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("shape,groups", ONE_LAUNCH + SPLIT)
def test_scratch_of_aligned_operands(dtype, shape, groups):
    forward, gradient = te.ep_group_norm_workspace_size, te.ep_group_norm_grad_workspace_size
    small = (shape, groups) in ONE_LAUNCH
    assert (forward(dtype, shape, groups, aligned=True) == 0) == small
    for size in (forward, gradient):
        assert size(dtype, shape, groups, aligned=True) <= size(dtype, shape, groups)
    # the gradient's, where it has one pass too (a sample up to 2048 fragments of 16 bytes): the channels'
    # sums alone, 8 bytes a channel for up to 8 blocks on each of 152 SMs
    if small and shape[1] * shape[2] * (4 if dtype == torch.float32 else 2) <= 2048 * 16:
        assert gradient(dtype, shape, groups, aligned=True) <= 8 * shape[-1] * min(shape[0], 8 * 152)


REFUSALS = """
import ctypes, json, sys
sys.path.insert(0, %r)
from transformer_epilogue_gb300 import _binding
lib = _binding.load_library()
A, B, C, D, E, F, G, H, I = (0x7F0000000000 + i * (1 << 36) for i in range(9))
out = []
for shape, groups in %r:
    s = (ctypes.c_int64 * 3)(*shape)
    need = lib.ep_group_norm_workspace_size(1, s, groups)
    need_grad = lib.ep_group_norm_grad_workspace_size_aligned(1, s, groups)
    gn = lambda x, y, ws=None, n=0: lib.ep_group_norm(1, x, s, B, C, groups, 1e-5, 0, y, None, None, ws, n, None)
    gng = lambda x, n: lib.ep_group_norm_grad(1, A, x, s, B, C, groups, 0, D, E, F, G, H, I, n, None)
    out.append([gn(A, D), gn(A + 2, D + 2), gn(A, D + 2), gn(A + 2, D + 2, E, need), gn(A, D + 2, E, need),
                gng(I + (1 << 36), need_grad), gng(I + (1 << 36), max(0, need_grad - 16))])
print(json.dumps(out))
"""


def test_calls_are_refused_only_for_scratch_that_they_use():
    # (no device: a call that passes the checks ends in the device query, EP_ERR_CUDA)
    code = REFUSALS % (ROOT, ONE_LAUNCH)
    p = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, CUDA_VISIBLE_DEVICES=""), capture_output=True,
                       text=True, timeout=300, cwd=ROOT)
    assert p.returncode == 0, p.stderr[-2000:]
    workspace, passed = te.EP_ERR_WORKSPACE, te.EP_ERR_CUDA
    for case, got in zip(ONE_LAUNCH, json.loads(p.stdout)):
        assert got == [passed, workspace, workspace, passed, passed, passed, workspace], case


@pytest.mark.gpu
@pytest.mark.parametrize("shape,groups", ONE_LAUNCH)
def test_one_launch_without_scratch(lib, shape, groups):
    x = torch.randn(shape, device="cuda", dtype=torch.float16)
    g = torch.ones(shape[-1], device="cuda", dtype=torch.float16)
    ws = torch.full((te.ep_group_norm_workspace_size(x.dtype, shape, groups) + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    n0 = te.kernel_launch_count()
    y, _, _ = te.ep_group_norm(x, g, None, groups, workspace=ws)
    assert te.kernel_launch_count() == n0 + 1
    assert bool((ws == 0xA5).all()), "scratch written by a call that needs none"
    assert torch.equal(y, te.ep_group_norm(x, g, None, groups)[0])
    assert torch.equal(y, te.ep_group_norm(x, g, None, groups, workspace=ws[:0])[0])
