"""A feed-forward block from the operators together, forward and backward with its
activations kept in 8 bits, each step against the oracle on what it was given; the same
run captured, on other streams, twice at once and repeated."""
import numpy as np
import pytest
import torch

from oracle import products as op
from tests._helpers import U32
from tests._products import DT, HALF, assert_mx8, assert_within, f64, mx8_f64, y_delta, z_delta

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def block_inputs(rows, hidden, inner, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = DT[dtype]

    def n(*d, std=1.0):
        return (torch.randn(*d, device="cuda", generator=g) * std).to(t)

    return dict(x=n(rows, hidden), skip=n(rows, hidden, std=0.5), gamma=(n(hidden) * 0.2 + 1).to(t),
                w1=n(inner, hidden, std=hidden ** -0.5), b1=n(inner, std=0.1), w2=n(hidden, inner, std=inner ** -0.5),
                b2=n(hidden, std=0.1), dy=n(rows, hidden, std=0.5))


def run_block(lib, p, stream=None):
    """sum = x + skip; y = sum + W2 quick_gelu(W1 norm(sum) + b1) + b2, and back."""
    act = lib.EP_ACT_QUICK_GELU
    k = dict(stream=stream)
    t = p["x"].dtype
    w1, s1 = lib.ep_quantize_mx8(p["w1"], **k)
    w2, s2 = lib.ep_quantize_mx8(p["w2"], **k)
    q, qs, total, inv = lib.ep_skip_rms_norm_mx8(p["x"], p["skip"], p["gamma"], input_skip_bias_sum=True, inv_std_dev=True, **k)
    h, z, zs = lib.ep_matmul_bias_act(q, w1, p["b1"], activation=act, A_scales=qs, W_scales=s1, dtype=t, Z=E4M3, **k)
    hq, hs = lib.ep_quantize_mx8(h, **k)
    y, _, _ = lib.ep_matmul_bias_act(hq, w2, p["b2"], total, A_scales=hs, W_scales=s2, **k)
    dh, dw2, db2 = lib.ep_matmul_bias_act_grad(p["dy"], hq, p["w2"], A_scales=hs, dbias=True, **k)
    dn, dw1, db1 = lib.ep_matmul_bias_act_grad(dh, q, p["w1"], z, act, A_scales=qs, Z_scales=zs, dbias=True, **k)
    dx, dg, _ = lib.ep_skip_rms_norm_grad(dn, total, p["gamma"], inv, dsum=p["dy"], **k)
    return dict(w1=(w1, s1), w2=(w2, s2), q=(q, qs), total=total, inv=inv, h=h, z=(z, zs), hq=(hq, hs), y=y, dh=dh, dw2=dw2,
                db2=db2, dn=dn, dw1=dw1, db1=db1, dx=dx, dg=dg)


def leaves(out):
    for k in sorted(out):
        for v in out[k] if isinstance(out[k], tuple) else (out[k],):
            yield k, v.view(torch.uint8) if v.element_size() == 1 else v


def assert_same(a, b):
    for (k, u), (_, v) in zip(leaves(a), leaves(b)):
        assert torch.equal(u, v), k


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,hidden,inner", [(1, 64, 96), (37, 256, 1000), (9, 77, 130), (1100, 256, 1304)])
def test_block(lib, rows, hidden, inner, dtype):
    p = block_inputs(rows, hidden, inner, dtype, 31)
    o = run_block(lib, p)
    t = DT[dtype]
    half, slope = HALF[t], 64 * U32
    low = 2.0 ** -25 if dtype == "f16" else 0.0
    w1, w2 = mx8_f64(*o["w1"]), mx8_f64(*o["w2"])
    np.testing.assert_array_equal(w1, op.mx8_values(*op.mx8_quantize(f64(p["w1"]))))
    n = op.rms_norm(f64(p["x"]), f64(p["skip"]), f64(p["gamma"]), None, lib.DEFAULT_EPSILON)
    assert_mx8(*o["q"], n["y"], 200 * U32 * np.abs(n["y"]) + 4 * U32 * n["terms"] * n["inv"] * np.abs(f64(p["gamma"])), "block norm")
    a = mx8_f64(*o["q"])
    m1 = op.matmul(a, w1, f64(p["b1"]), None, "quick_gelu")
    d1 = z_delta(hidden, m1["z_scale"])
    assert_within(o["h"], m1["y"], y_delta(m1["z"], m1["y"], d1, "quick_gelu", 1.702), "block h")
    assert_mx8(*o["z"], m1["z"], d1, "block z")
    np.testing.assert_array_equal(mx8_f64(*o["hq"]), op.mx8_values(*op.mx8_quantize(f64(o["h"]))))
    h = mx8_f64(*o["hq"])
    m2 = op.matmul(h, w2, f64(p["b2"]), f64(o["total"]))
    assert_within(o["y"], m2["y"], z_delta(inner, m2["z_scale"]) + U32 * (np.abs(f64(o["total"])) + np.abs(m2["y"])), "block y")
    g2 = op.matmul_grad(f64(p["dy"]), h, f64(p["w2"]))
    assert_within(o["dh"], g2["dA"], z_delta(hidden, g2["dA_scale"]), "block dh")
    assert_within(o["dw2"], g2["dW"], z_delta(rows, g2["dW_scale"]), "block dw2")
    assert_within(o["db2"], g2["dbias"], 128 * U32 * g2["dbias_scale"], "block db2")
    g1 = op.matmul_grad(f64(o["dh"]), a, f64(p["w1"]), mx8_f64(*o["z"]), "quick_gelu")
    assert_within(o["dn"], g1["dA"], (half + slope) * g1["dA_scale"] + low * np.abs(f64(p["w1"])).sum(0) + z_delta(inner, g1["dA_scale"]),
                  "block dn")
    assert_within(o["dw1"], g1["dW"], (half + slope) * g1["dW_scale"] + low * np.abs(a).sum(0) + z_delta(rows, g1["dW_scale"]), "block dw1")
    assert_within(o["db1"], g1["dbias"], (slope + 128 * U32) * g1["dbias_scale"], "block db1")
    gn = op.rms_norm_grad(f64(o["dn"]), f64(o["total"]), f64(p["gamma"]), f64(o["inv"]), f64(p["dy"]))
    assert_within(o["dx"], gn["dX"], 64 * U32 * gn["dX_scale"], "block dx")
    assert_within(o["dg"], gn["dgamma"], 128 * U32 * gn["dgamma_scale"], "block dgamma")


@pytest.mark.parametrize("rows,hidden,inner", [(37, 256, 1000), (1100, 257, 1304)])
def test_block_captured_and_repeated(lib, rows, hidden, inner):
    """A captured run gives the eager run's bits on the inputs of each replay; so does another eager run."""
    p, other = block_inputs(rows, hidden, inner, "bf16", 32), block_inputs(rows, hidden, inner, "bf16", 33)
    first, second = run_block(lib, p), run_block(lib, other)
    assert_same(first, run_block(lib, p))
    held = {k: v.clone() for k, v in p.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_block(lib, held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run_block(lib, held)
    for want, inputs in ((first, p), (second, other), (first, p)):
        for k, v in inputs.items():
            held[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert_same(want, got)
    assert lib.ep_pipeline_timeouts() == 0


def test_two_streams_at_once(lib):
    """Runs on two streams, given by argument and as the current one, next to each other."""
    a, b = block_inputs(700, 512, 2048, "f16", 34), block_inputs(50, 768, 1000, "f16", 35)
    want_a, want_b = run_block(lib, a), run_block(lib, b)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    t.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(8):
        ga = run_block(lib, a, stream=s)
        with torch.cuda.stream(t):
            gb = run_block(lib, b)
        got.append((ga, gb))
    torch.cuda.synchronize()
    for ga, gb in got:
        assert_same(want_a, ga)
        assert_same(want_b, gb)
    assert lib.ep_pipeline_timeouts() == 0


@pytest.mark.parametrize("m,n,k,off", [(7, 40, 64, 0), (7, 39, 64, 0), (130, 264, 72, 1), (1040, 2568, 64, 0), (1040, 2563, 64, 1)])
def test_nothing_behind_the_outputs(lib, m, n, k, off):
    """Y, Z (16 and 8 bits), its scales and the gradients leave what lies around them alone."""
    g = torch.Generator(device="cuda").manual_seed(36)
    t = torch.bfloat16
    a, w, b, r = (torch.randn(*d, device="cuda", generator=g).to(t) for d in ((m, k), (n, k), (n,), (m, n)))

    def guarded(shape, dtype):
        size = torch.Size(shape).numel()
        raw = torch.full((size + 512 + off,), 90, dtype=torch.uint8, device="cuda") if dtype.itemsize == 1 else \
            torch.full((size + 512 + off,), 7.0, dtype=dtype, device="cuda")
        return raw, raw[256 + off:256 + off + size].view(dtype).view(shape)

    def untouched(raw, inner):
        lo = 256 + off
        hi = lo + inner.numel()
        v = 90 if raw.dtype is torch.uint8 else 7.0
        assert (raw[:lo] == v).all() and (raw[hi:] == v).all()

    y0, z0, _ = lib.ep_matmul_bias_act(a, w, b, r, lib.EP_ACT_SILU, Z=True)
    _, q0, s0 = lib.ep_matmul_bias_act(a, w, b, r, lib.EP_ACT_SILU, Z=E4M3)
    ry, y = guarded((m, n), t)
    rz, z = guarded((m, n), t)
    rq, q = guarded((m, n), E4M3)
    rs, s = guarded((m, -(-n // 32)), torch.float8_e8m0fnu)
    lib.ep_matmul_bias_act(a, w, b, r, lib.EP_ACT_SILU, Y=y, Z=z)
    assert torch.equal(y, y0) and torch.equal(z, z0)
    lib.ep_matmul_bias_act(a, w, b, r, lib.EP_ACT_SILU, Y=y, Z=q, Z_scales=s)
    assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s.view(torch.uint8), s0.view(torch.uint8))
    want = lib.ep_matmul_bias_act_grad(r, a, w, z0, lib.EP_ACT_SILU, dbias=True)
    pairs = [guarded(x.shape, t) for x in want]
    lib.ep_matmul_bias_act_grad(r, a, w, z0, lib.EP_ACT_SILU, dA=pairs[0][1], dW=pairs[1][1], dbias=pairs[2][1])
    for (raw, got), x in zip(pairs, want):
        assert torch.equal(got, x)
        untouched(raw, got)
    for raw, x in ((ry, y), (rz, z), (rq, q), (rs, s)):
        untouched(raw, x)


def test_given_workspace_is_enough(lib):
    """Workspaces of exactly the sizes asked for, whatever they hold."""
    for m, n, k, off in ((70, 130, 63, 0), (70, 136, 64, 1), (1040, 2568, 256, 0)):
        g = torch.Generator(device="cuda").manual_seed(37)
        t = torch.float16
        a, w, r = (torch.randn(*d, device="cuda", generator=g).to(t) for d in ((m, k), (n, k), (m, n)))
        z = r.clone()
        if off:
            a, w = (torch.cat([x.view(-1)[:1], x.view(-1)])[1:].view(x.shape) for x in (a, w))
        (qa, sa), (qw, sw) = lib.ep_quantize_mx8(a), lib.ep_quantize_mx8(w)
        calls = [(lib.ep_matmul_bias_act_workspace_size(a.shape, w.shape, aligned=not off),
                  lambda ws: lib.ep_matmul_bias_act(a, w, workspace=ws)[:1]),
                 (lib.ep_matmul_bias_act_workspace_size(a.shape, w.shape, mx8=True, aligned=True),
                  lambda ws: lib.ep_matmul_bias_act(qa, qw, A_scales=sa, W_scales=sw, dtype=t, workspace=ws)[:1]),
                 (lib.ep_matmul_bias_act_grad_workspace_size(a.shape, w.shape, lib.EP_ACT_GELU, aligned=not off),
                  lambda ws: lib.ep_matmul_bias_act_grad(r, a, w, z, lib.EP_ACT_GELU, dbias=True, workspace=ws)),
                 (lib.ep_skip_rms_norm_grad_workspace_size(t, a.shape),
                  lambda ws: lib.ep_skip_rms_norm_grad(a, a, a[0].clone(), torch.ones(m, 1, device="cuda"), dbias=True, workspace=ws))]
        for need, call in calls:
            want = call(None)
            raw = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")  # (NaN as 16-bit and 32-bit numbers)
            got = call(raw[:need] if need else None)
            assert all(torch.equal(x, y) for x, y in zip(want, got))
            assert (raw[need:] == 255).all()
