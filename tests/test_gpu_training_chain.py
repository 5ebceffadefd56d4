"""The operators run together as a training step uses them, eagerly and from a
captured graph.

The channels-last block: group norm + SiLU -> dropout -> bias + residual
(BiasAdd), then its gradient.  The token block: BiasSoftmax -> dropout in
place; dropout(x + bias) + residual -> SkipLayerNormalization.  Every
intermediate is compared with the oracle on the values that the step before
left, so each operator's bound is its own.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import training as tr
from tests._helpers import U32, assert_norm_close
from tests._training import assert_within, dropout_inputs, group_norm_inputs, norm_delta

pytestmark = pytest.mark.gpu

RATIO, SEED = 0.2, 77


def block(lib, t, groups, step):
    """Forward and gradient of the channels-last block; everything it made."""
    silu = lib.EP_ACT_SILU
    y, mean, inv = lib.ep_group_norm(t["X"], t["gamma"], t["beta"], groups, 1e-5, silu, mean=True, inv_std_dev=True)
    z = lib.ep_bias_dropout(y, RATIO, SEED, 1, offset_device=step)
    out = lib.ep_bias_add(z, t["bias"], t["skip"])
    dz, dbias = lib.ep_bias_dropout_grad(t["dY"], RATIO, SEED, 1, offset_device=step, dbias=True)
    dx, dgamma, dbeta = lib.ep_group_norm_grad(dz, t["X"], t["gamma"], t["beta"], mean, inv, groups, silu)
    return dict(y=y, mean=mean, inv=inv, z=z, out=out, dz=dz, dbias=dbias, dx=dx, dgamma=dgamma, dbeta=dbeta)


def block_inputs(shape, dtype, seed):
    d = group_norm_inputs(shape, dtype, seed)
    g = torch.Generator().manual_seed(seed + 1)
    d["bias"] = torch.randn(shape[-1], generator=g).mul(0.1).to(d["X"].dtype)
    d["skip"] = torch.randn(shape, generator=g).to(d["X"].dtype)
    return d


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape,groups", [((2, 256, 320), 32), ((2, 37, 189), 9), ((64, 1, 512), 8)])
def test_channels_last_block(lib, dtype, shape, groups):
    d = block_inputs(shape, dtype, 5)
    step = torch.tensor([3], dtype=torch.int64, device="cuda")
    r = {k: v.cpu() for k, v in block(lib, {k: v.cuda() for k, v in d.items()}, groups, step).items()}
    c = shape[-1]
    f = tr.group_norm(d["X"], d["gamma"], d["beta"], groups, 1e-5, True)
    assert_within(r["y"], f["Y"], norm_delta(f["mean"], f["inv_std_dev"], d["gamma"], groups, c), "chain y")
    z = tr.bias_dropout(r["y"], RATIO, SEED, 4)
    assert_within(r["z"], z["Y"], 4 * U32 * np.abs(z["Y"]), "chain z")
    o = oracle.bias_add(r["z"], d["bias"], d["skip"])
    mag = np.abs(oracle.bias_add(r["z"].abs(), d["bias"].abs(), d["skip"].abs()))
    assert_within(r["out"], o.reshape(shape), 4 * U32 * mag.reshape(shape), "chain out")
    dz = tr.bias_dropout_grad(d["dY"], RATIO, SEED, 4)
    assert_within(r["dz"], dz["dX"], 2 * U32 * np.abs(dz["dX"]), "chain dz")
    assert_within(r["dbias"], dz["dbias"], 64 * U32 * dz["dbias_scale"], "chain dbias")
    g = tr.group_norm_grad(r["dz"], d["X"], d["gamma"], d["beta"], r["mean"], r["inv"], groups, True)
    assert_within(r["dx"], g["dX"], 64 * U32 * g["dX_scale"], "chain dx")
    assert_within(r["dgamma"], g["dgamma"], 64 * U32 * g["dgamma_scale"], "chain dgamma")
    assert_within(r["dbeta"], g["dbeta"], 64 * U32 * g["dbeta_scale"], "chain dbeta")


@pytest.mark.parametrize("shape,groups", [((2, 1000, 96), 8), ((300, 1, 256), 4)])
def test_block_from_a_captured_graph(lib, shape, groups):
    d = block_inputs(shape, "bf16", 9)
    t = {k: v.cuda() for k, v in d.items()}
    step = torch.tensor([0], dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block(lib, t, groups, step)   # warm-up
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(lib, t, groups, step)
    masks = []
    for k in (0, 1, 5):
        step.fill_(k)
        t["X"].copy_(d["X"] * (1 + k))   # other inputs on every replay
        graph.replay()
        torch.cuda.synchronize()
        got_k = {n: v.clone() for n, v in got.items()}
        want = block(lib, t, groups, step)
        for n in want:
            assert torch.equal(got_k[n], want[n]), (k, n)
        masks.append(got_k["dz"] != 0)
    assert not torch.equal(masks[0], masks[1]) and not torch.equal(masks[1], masks[2])


def test_two_streams_at_once(lib):
    # calls that overlap on the GPU, each with scratch of its own
    ds = [block_inputs((2, 3000, 64), "f16", 100 + k) for k in range(2)]
    ts = [{k: v.cuda() for k, v in d.items()} for d in ds]
    step = torch.tensor([0], dtype=torch.int64, device="cuda")
    want = [block(lib, t, 4, step) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    got = [None, None]
    for _ in range(10):
        for i, (s, t) in enumerate(zip(streams, ts)):
            with torch.cuda.stream(s):
                got[i] = block(lib, t, 4, step)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_attention_probabilities_and_block_end(lib):
    g = torch.Generator().manual_seed(3)
    scores = (torch.randn(2, 4, 32, 96, generator=g) * 2).half()
    mask = torch.zeros(2, 32, 96, dtype=torch.float16)
    p = lib.ep_bias_softmax(scores.cuda(), mask.cuda(), axis=3, is_inner_broadcast=1)
    before = p.cpu()
    lib.ep_bias_dropout(p, RATIO, SEED, 2, Y=p)
    o = tr.bias_dropout(before, RATIO, SEED, 2)
    assert_within(p.cpu(), o["Y"], 4 * U32 * np.abs(o["Y"]), "dropped probabilities")

    d = dropout_inputs((3, 50, 256), "f16", 4)
    h = lib.ep_bias_dropout(d["X"].cuda(), RATIO, SEED, 3, bias=d["bias"].cuda(), residual=d["residual"].cuda())
    w = torch.ones(256, dtype=torch.float16)
    y, _ = lib.ep_skip_layer_norm(h, d["residual"].cuda(), w.cuda(), epsilon=1e-5)
    o = tr.bias_dropout(d["X"], RATIO, SEED, 3, d["bias"], d["residual"])
    assert_within(h.cpu(), o["Y"], U32 * (3 * np.abs(o["kept"]) + np.abs(o["Y"])), "block end")
    ln = oracle.skip_layer_norm(h.cpu(), d["residual"], w, epsilon=1e-5)["output"]
    assert_norm_close(y.cpu(), ln, torch.float16)
