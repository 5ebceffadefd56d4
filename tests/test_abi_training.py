"""Refusals of GroupNorm and BiasDropout: the C entry points' (in a process
without a device) and the binding's (no GPU needed)."""
import json
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def built():
    from transformer_epilogue_gb300 import build
    build.build()


def test_host_validation_contracts(built):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    p = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "abi_training_cases.py")], env=env,
                       capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert p.returncode == 0, p.stdout[-4000:] + p.stderr[-4000:]
    res = json.loads(p.stdout.strip().splitlines()[-1])
    assert res["cases"] >= 90 and not res["failures"]


def test_binding_refuses_host_tensors(built):
    import transformer_epilogue_gb300 as te
    x, g = torch.zeros(2, 3, 8), torch.ones(8)
    for call in (lambda: te.ep_group_norm(x, g, g, 2), lambda: te.ep_group_norm_grad(x, x, g, g, x, x, 2),
                 lambda: te.ep_bias_dropout(x, 0.1, 1), lambda: te.ep_bias_dropout_grad(x, 0.1, 1),
                 lambda: te.ep_group_norm(None, g, g, 2), lambda: te.ep_group_norm(x, g, g)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_refusals(lib):
    x = torch.randn(2, 6, 8, device="cuda", dtype=torch.float16)
    g = torch.ones(8, device="cuda", dtype=torch.float16)
    _, m, i = lib.ep_group_norm(x, g, g, 2, mean=True, inv_std_dev=True)
    f32 = torch.float32
    refused = [
        lambda: lib.ep_group_norm(x.double(), g.double(), None, 2),
        lambda: lib.ep_group_norm(x, g.float(), None, 2),
        lambda: lib.ep_group_norm(x, g[:4], None, 2),
        lambda: lib.ep_group_norm(x, g.cpu(), None, 2),
        lambda: lib.ep_group_norm(x.transpose(1, 2), g, None, 2),
        lambda: lib.ep_group_norm(x[:, 0], g, None, 2),
        lambda: lib.ep_group_norm(x, g, None, 2, mean=torch.empty(2, 2, device="cuda", dtype=torch.float16)),
        lambda: lib.ep_group_norm(x, g, None, 2, mean=torch.empty(3, device="cuda", dtype=f32)),
        lambda: lib.ep_group_norm(x, g, None, 2, Y=torch.empty(2, 6, 4, device="cuda", dtype=torch.float16)),
        lambda: lib.ep_group_norm_grad(x.float(), x, g, g, m, i, 2),
        lambda: lib.ep_group_norm_grad(x[:1], x, g, g, m, i, 2),
        lambda: lib.ep_group_norm_grad(x, x, g, g, m[:1], i, 2),
        lambda: lib.ep_group_norm_grad(x, x, g, g, None, i, 2),
        lambda: lib.ep_group_norm_grad(x, x, g, g, True, i, 2),
        lambda: lib.ep_group_norm_grad(x, x, g, g, m, i, 2, dgamma=torch.empty(8, device="cuda", dtype=f32)),
        lambda: lib.ep_bias_dropout(x, 0.1, -1),
        lambda: lib.ep_bias_dropout(x, 0.1, 1 << 64),
        lambda: lib.ep_bias_dropout(x, 0.1, 1, bias=g[:4]),
        lambda: lib.ep_bias_dropout(x, 0.1, 1, residual=x[:1]),
        lambda: lib.ep_bias_dropout(x, 0.1, 1, residual=x.float()),
        lambda: lib.ep_bias_dropout(x, 0.1, 1, offset_device=torch.zeros(2, dtype=torch.int64, device="cuda")),
        lambda: lib.ep_bias_dropout(x, 0.1, 1, offset_device=torch.zeros(1, dtype=torch.int64)),
        lambda: lib.ep_bias_dropout(x, 0.1, 1, offset_device=torch.zeros(1, dtype=f32, device="cuda")),
        lambda: lib.ep_bias_dropout_grad(x, 0.1, 1, dbias=torch.empty(4, device="cuda", dtype=torch.float16)),
        lambda: lib.ep_bias_dropout_grad(x, 0.1, 1, dX=x[:1]),
    ]
    n0 = lib.kernel_launch_count()
    for k, call in enumerate(refused):
        with pytest.raises((ValueError, TypeError)):
            call()
    for k, call in enumerate((lambda: lib.ep_group_norm(x, g, None, 3), lambda: lib.ep_group_norm(x, g, None, 0),
                              lambda: lib.ep_group_norm(x, g, None, 2, -1.0),
                              lambda: lib.ep_group_norm(x, g, None, 2, activation=5),
                              lambda: lib.ep_bias_dropout(x, 1.0, 1))):
        with pytest.raises(lib.EpError) as e:
            call()
        assert e.value.status == lib.EP_ERR_INVALID_ARG, k
    assert lib.kernel_launch_count() == n0
