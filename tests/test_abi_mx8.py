"""Refusals of MX8 rows, the RMS norm and the matrix product: the C entry points' (in a
process without a device) and the binding's."""
import json
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module")
def built():
    from transformer_epilogue_gb300 import build
    build.build()


def test_host_validation_contracts(built):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    p = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "abi_mx8_cases.py")], env=env, capture_output=True,
                       text=True, timeout=300, cwd=ROOT)
    assert p.returncode == 0, p.stdout[-4000:] + p.stderr[-4000:]
    res = json.loads(p.stdout.strip().splitlines()[-1])
    assert res["cases"] >= 140 and not res["failures"] and res["launches"] == 0, res


def test_binding_refuses_host_tensors(built):
    import transformer_epilogue_gb300 as te
    x, g, w = torch.zeros(3, 8), torch.ones(8), torch.zeros(4, 8)
    q, s = torch.zeros(3, 8, dtype=E4M3), torch.zeros(3, 1, dtype=E8M0)
    for call in (lambda: te.ep_quantize_mx8(x), lambda: te.ep_dequantize_mx8(q, s, torch.float32),
                 lambda: te.ep_skip_rms_norm_mx8(x, x, g), lambda: te.ep_skip_rms_norm_grad(x, x, g, x[:, :1]),
                 lambda: te.ep_matmul_bias_act(x.half(), w.half()), lambda: te.ep_matmul_bias_act_grad(x.half(), x.half(), w.half()),
                 lambda: te.ep_quantize_mx8(None), lambda: te.ep_matmul_bias_act(None, w)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_refusals(lib):
    t = torch.float16
    x, g = torch.randn(4, 40, device="cuda", dtype=t), torch.ones(40, device="cuda", dtype=t)
    w, b, r = (torch.randn(*d, device="cuda", dtype=t) for d in ((24, 40), (24,), (4, 24)))
    q, s = lib.ep_quantize_mx8(x)
    qw, sw = lib.ep_quantize_mx8(w)
    inv = torch.ones(4, 1, device="cuda")
    dy = torch.randn(4, 24, device="cuda", dtype=t)
    refused = [
        lambda: lib.ep_quantize_mx8(x.double()), lambda: lib.ep_quantize_mx8(x.t()), lambda: lib.ep_quantize_mx8(x[0, 0]),
        lambda: lib.ep_quantize_mx8(x, Q=q), lambda: lib.ep_quantize_mx8(x, scales=s), lambda: lib.ep_quantize_mx8(x, q, s[:2]),
        lambda: lib.ep_quantize_mx8(x, q.view(torch.uint8), s), lambda: lib.ep_dequantize_mx8(q, s),
        lambda: lib.ep_dequantize_mx8(q, s[:, :1], t), lambda: lib.ep_dequantize_mx8(q, s, torch.int32),
        lambda: lib.ep_dequantize_mx8(q, s, t, Y=torch.empty(4, 40, device="cuda")), lambda: lib.ep_dequantize_mx8(x, s, t),
        lambda: lib.ep_skip_rms_norm_mx8(x, x[:1], g), lambda: lib.ep_skip_rms_norm_mx8(x, x, g[:8]),
        lambda: lib.ep_skip_rms_norm_mx8(x, x.float(), g), lambda: lib.ep_skip_rms_norm_mx8(x, x, None),
        lambda: lib.ep_skip_rms_norm_mx8(x, x, g, inv_std_dev=torch.empty(3, device="cuda")),
        lambda: lib.ep_skip_rms_norm_mx8(x, x, g, inv_std_dev=torch.empty(4, device="cuda", dtype=t)),
        lambda: lib.ep_skip_rms_norm_mx8(x, x, g, epsilon=-1.0), lambda: lib.ep_skip_rms_norm_mx8(x, x.cpu(), g),
        lambda: lib.ep_skip_rms_norm_mx8(x[:, :0], None, g[:0]),
        lambda: lib.ep_skip_rms_norm_grad(x, x, g, None), lambda: lib.ep_skip_rms_norm_grad(x, x[:2], g, inv),
        lambda: lib.ep_skip_rms_norm_grad(x, x, g, inv[:2]), lambda: lib.ep_skip_rms_norm_grad(x, x, g, inv, dsum=x.float()),
        lambda: lib.ep_skip_rms_norm_grad(x, x, g, inv, dgamma=b), lambda: lib.ep_skip_rms_norm_grad(x, x, g, inv, dX=x[:2]),
        lambda: lib.ep_matmul_bias_act(x.float(), w.float()), lambda: lib.ep_matmul_bias_act(x, w.float()),
        lambda: lib.ep_matmul_bias_act(x, w[:, :8].contiguous()), lambda: lib.ep_matmul_bias_act(x, w[0]),
        lambda: lib.ep_matmul_bias_act(x, w.t()), lambda: lib.ep_matmul_bias_act(x, w, b[:8]),
        lambda: lib.ep_matmul_bias_act(x, w, b, r[:2]), lambda: lib.ep_matmul_bias_act(x, w, activation=6),
        lambda: lib.ep_matmul_bias_act(x, w, alpha=float("nan")), lambda: lib.ep_matmul_bias_act(x, w, A_scales=s),
        lambda: lib.ep_matmul_bias_act(x, w, dtype=torch.bfloat16), lambda: lib.ep_matmul_bias_act(x, w, Z=torch.float32),
        lambda: lib.ep_matmul_bias_act(x, w, Z=torch.empty(4, 24, device="cuda", dtype=E4M3)),
        lambda: lib.ep_matmul_bias_act(x, w, Z_scales=s), lambda: lib.ep_matmul_bias_act(q, qw, A_scales=s, W_scales=sw),
        lambda: lib.ep_matmul_bias_act(q, qw, A_scales=s, W_scales=sw, dtype=torch.float32),
        lambda: lib.ep_matmul_bias_act(q, qw, A_scales=s, dtype=t), lambda: lib.ep_matmul_bias_act(q, w, A_scales=s, dtype=t),
        lambda: lib.ep_matmul_bias_act(x, w, workspace=torch.empty(16, dtype=torch.uint8)),
        lambda: lib.ep_matmul_bias_act_grad(dy, x, w, activation=1), lambda: lib.ep_matmul_bias_act_grad(dy[:2], x, w),
        lambda: lib.ep_matmul_bias_act_grad(dy, x, w.bfloat16()), lambda: lib.ep_matmul_bias_act_grad(dy, q, w),
        lambda: lib.ep_matmul_bias_act_grad(dy, x, w, A_scales=s), lambda: lib.ep_matmul_bias_act_grad(dy, x, w, Z=x, activation=1),
        lambda: lib.ep_matmul_bias_act_grad(dy, x, w, dA=dy), lambda: lib.ep_matmul_bias_act_grad(dy, x, w, dbias=g),
        lambda: lib.ep_matmul_bias_act_grad(dy, x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
    ]
    before = lib.kernel_launch_count()
    for i, call in enumerate(refused):
        with pytest.raises((ValueError, TypeError, lib.EpError)):
            call()
            pytest.fail(f"call {i} was not refused")
    assert lib.kernel_launch_count() == before
