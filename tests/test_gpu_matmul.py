"""The matrix product with its epilogue, and its gradient, against the float64 oracle."""
import time

import numpy as np
import pytest
import torch

from oracle import products as op
from tests._helpers import U32
from tests._products import (DT, HALF, assert_mx8, assert_within, at_offset, cuda, f64, mx8_f64, product_inputs, y_delta,
                             z_delta)

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def act_code(lib, act):
    return getattr(lib, "EP_ACT_" + act.upper())


def forward(lib, m, n, k, dtype, act="none", bias=True, residual=True, save=None, mx8=False, off=0, seed=1, alpha=1.702):
    a, w, b, r = product_inputs(m, n, k, dtype, seed, bias, residual)
    da, dw, db, dr = cuda(a, w, b, r)
    kw = {}
    if mx8:
        (da, sa), (dw, sw) = lib.ep_quantize_mx8(da), lib.ep_quantize_mx8(dw)
        a64, w64 = mx8_f64(da, sa), mx8_f64(dw, sw)
        kw = dict(A_scales=sa, W_scales=sw, dtype=DT[dtype])
    else:
        a64, w64 = f64(a), f64(w)
    if off:
        da, dw, db, dr = (at_offset(t, off) for t in (da, dw, db, dr))
        if mx8:
            kw.update(A_scales=at_offset(sa, off), W_scales=at_offset(sw, off))
    y, z, zs = lib.ep_matmul_bias_act(da, dw, db, dr, act_code(lib, act), alpha, Z={None: None, "t": True, "mx8": E4M3}[save],
                                      **kw)
    o = op.matmul(a64, w64, f64(b), f64(r), act, alpha)
    zd = z_delta(k, o["z_scale"])
    yd = y_delta(o["z"], op.activation(o["z"], act, alpha), zd, act, alpha)
    if residual:
        yd = yd + U32 * (np.abs(f64(r)) + np.abs(o["y"]))
    assert_within(y, o["y"], yd, "mm y")
    if save == "t":
        assert zs is None
        assert_within(z, o["z"], zd, "mm z")
    elif save == "mx8":
        assert_mx8(z, zs, o["z"], zd, "mm z8")
    else:
        assert z is None and zs is None


# one K tile, a ragged one, several; one row to several tiles of rows; ragged columns
SPLIT = [(1, 128, 64), (1, 1, 1), (2, 8, 8), (7, 130, 72), (16, 256, 1024), (17, 96, 200), (33, 384, 4096), (64, 64, 640),
         (65, 1000, 333), (100, 520, 129), (128, 2048, 512), (200, 136, 264), (300, 31, 1001)]
# enough tiles for pairs of CTAs
PAIR = [(1024, 2560, 64), (1100, 2600, 200), (2049, 1288, 1000), (4100, 520, 72)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("mnk", SPLIT, ids=str)
def test_few_tiles(lib, mnk, dtype):
    forward(lib, *mnk, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("mnk", SPLIT, ids=str)
def test_few_tiles_mx8(lib, mnk, dtype):
    forward(lib, *mnk, dtype, mx8=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("mnk", PAIR, ids=str)
def test_many_tiles(lib, mnk, dtype):
    forward(lib, *mnk, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("mnk", PAIR, ids=str)
def test_many_tiles_mx8(lib, mnk, dtype):
    forward(lib, *mnk, dtype, mx8=True)


@pytest.mark.parametrize("mx8", [False, True])
@pytest.mark.parametrize("save", [None, "t", "mx8"])
@pytest.mark.parametrize("act", op.ACTS)
@pytest.mark.parametrize("mnk", [(5, 72, 96), (9, 101, 40), (1040, 2568, 64), (1040, 2563, 48)], ids=str)
def test_epilogues(lib, mnk, act, save, mx8):
    forward(lib, *mnk, "bf16", act, save=save, mx8=mx8)


@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("mnk", [(5, 72, 96), (1040, 2568, 64)], ids=str)
def test_without(lib, mnk, bias, residual):
    forward(lib, *mnk, "f16", "quick_gelu", bias, residual, save="mx8", alpha=0.7)


@pytest.mark.parametrize("mx8", [False, True])
@pytest.mark.parametrize("off", [1, 8])
@pytest.mark.parametrize("mnk", [(5, 72, 96), (40, 136, 512), (1040, 2568, 64)], ids=str)
def test_alignments(lib, mnk, off, mx8):
    forward(lib, *mnk, "f16", "gelu", save="t", off=off, mx8=mx8)


def test_leading_dimensions_and_no_depth(lib):
    a, w, b, r = product_inputs(12, 40, 24, "bf16", 5)
    da, dw, db, dr = cuda(a, w, b, r)
    flat = lib.ep_matmul_bias_act(da, dw, db, dr)[0]
    assert torch.equal(lib.ep_matmul_bias_act(da.view(2, 6, 24), dw, db, dr.view(2, 6, 40))[0], flat.view(2, 6, 40))
    assert torch.equal(lib.ep_matmul_bias_act(da[0], dw, db, dr[0])[0], flat[0])
    e = torch.empty(12, 0, dtype=torch.bfloat16, device="cuda"), torch.empty(40, 0, dtype=torch.bfloat16, device="cuda")
    y, z, _ = lib.ep_matmul_bias_act(*e, db, dr, Z=True)
    assert torch.equal(z, db.expand(12, 40)) and torch.equal(y, (db.float() + dr.float()).to(torch.bfloat16))
    assert not lib.ep_matmul_bias_act(*e)[0].any()
    assert lib.ep_matmul_bias_act(da[:0], dw, db)[0].shape == (0, 40)
    assert lib.ep_matmul_bias_act(da, dw[:0])[0].shape == (12, 0)


def test_residual_in_place(lib):
    for m, n, k in ((9, 136, 64), (1040, 2568, 64)):
        a, w, b, r = cuda(*product_inputs(m, n, k, "f16", 6))
        want = lib.ep_matmul_bias_act(a, w, b, r, lib.EP_ACT_SILU)[0]
        lib.ep_matmul_bias_act(a, w, b, r, lib.EP_ACT_SILU, Y=r)
        assert torch.equal(r, want)


@pytest.mark.parametrize("act", op.ACTS)
@pytest.mark.parametrize("m", [3, 1040])
def test_large_and_infinite_values(lib, act, m):
    """A product with the identity: z = the bias exactly, from the smallest to infinity; NaN stays in its place."""
    n = 2568 if m > 100 else 72
    vals = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3.0, -3.0, 12.0, -12.0, 60.0, -60.0, 100.0, -100.0, 3e4, -3e4, 1e30, -1e30,
                         float("inf"), float("-inf"), float("nan")])
    b = vals[torch.arange(n) % len(vals)].to(torch.bfloat16)
    a, w = torch.zeros(m, 64, dtype=torch.bfloat16), torch.zeros(n, 64, dtype=torch.bfloat16)
    y, z, _ = lib.ep_matmul_bias_act(*cuda(a, w, b), activation=act_code(lib, act), Z=True)
    z64 = np.broadcast_to(f64(b), (m, n))
    np.testing.assert_array_equal(f64(z), z64)
    want = op.activation(z64, act)
    assert_within(y, want, y_delta(np.nan_to_num(z64, posinf=0, neginf=0), np.nan_to_num(want, posinf=0), 0.0, act, 1.702),
                  "mm limits")


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------

def backward(lib, m, n, k, dtype, act="quick_gelu", save="t", kept="t", off=0, seed=2, alpha=1.702, dbias=True):
    t = DT[dtype]
    a, w, b, r = product_inputs(m, n, k, dtype, seed)
    g = torch.Generator().manual_seed(seed + 1)
    dy = torch.randn(m, n, generator=g).to(t)
    z = (a.float() @ w.float().t() + b.float()).to(t)
    da, dw, dz, ddy = cuda(a, w, z, dy)
    kw, a64, z64 = {}, f64(a), f64(z)
    if kept == "mx8":
        da, kw["A_scales"] = lib.ep_quantize_mx8(da)
        a64 = mx8_f64(da, kw["A_scales"])
    if save == "mx8":
        dz, kw["Z_scales"] = lib.ep_quantize_mx8(dz)
        z64 = mx8_f64(dz, kw["Z_scales"])
    if off:
        da, dw, dz, ddy = (at_offset(x, off) for x in (da, dw, dz, ddy))
        kw = {name: at_offset(x, off) for name, x in kw.items()}
    ga, gw, gb = lib.ep_matmul_bias_act_grad(ddy, da, dw, dz if act != "none" else None, act_code(lib, act), alpha,
                                             dbias=True if dbias else None,
                                             **(kw if act != "none" else {x: v for x, v in kw.items() if x != "Z_scales"}))
    o = op.matmul_grad(f64(dy), a64, f64(w), z64, act, alpha)
    # where dz is a subnormal of float16, its rounding is off by half of 2^-24 whatever its size
    half, slope = (HALF[t] if act != "none" else 0.0), (64 * U32 if act != "none" else 0.0)
    low = 2.0 ** -25 if act != "none" and dtype == "f16" else 0.0
    assert_within(ga, o["dA"], (half + slope) * o["dA_scale"] + low * np.abs(f64(w)).sum(0) + z_delta(n, o["dA_scale"]), "mm dA")
    assert_within(gw, o["dW"], (half + slope) * o["dW_scale"] + low * np.abs(a64).sum(0) + z_delta(m, o["dW_scale"]), "mm dW")
    if dbias:
        assert_within(gb, o["dbias"], (slope + 128 * U32) * o["dbias_scale"], "mm dbias")


GRADS = [(1, 1, 1), (8, 8, 8), (3, 70, 130), (64, 128, 64), (129, 200, 72), (130, 136, 1001), (500, 33, 96), (1000, 777, 255),
         (2048, 1304, 1160), (1160, 2056, 2600)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("mnk", GRADS, ids=str)
def test_grad(lib, mnk, dtype):
    backward(lib, *mnk, dtype)


@pytest.mark.parametrize("save,kept", [("mx8", "t"), ("t", "mx8"), ("mx8", "mx8")])
@pytest.mark.parametrize("mnk", GRADS, ids=str)
def test_grad_from_checkpoints(lib, mnk, save, kept):
    backward(lib, *mnk, "bf16", "fast_gelu", save, kept)


@pytest.mark.parametrize("act", op.ACTS)
@pytest.mark.parametrize("save", ["t", "mx8"])
@pytest.mark.parametrize("mnk", [(70, 72, 96), (70, 73, 95)], ids=str)
def test_grad_activations(lib, mnk, act, save):
    backward(lib, *mnk, "f16", act, save, alpha=0.8, dbias=act != "relu")


@pytest.mark.parametrize("off", [1, 8])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("kept", ["t", "mx8"])
def test_grad_alignments(lib, off, act, kept):
    backward(lib, 130, 72, 96, "bf16", act, "mx8", kept, off=off)


def test_grad_parts_and_empty_sums(lib):
    a, w, b, dy = cuda(*product_inputs(70, 40, 24, "bf16", 8))
    full = lib.ep_matmul_bias_act_grad(dy, a, w, dbias=True)
    for i in range(3):
        want = [i == j for j in range(3)]
        got = lib.ep_matmul_bias_act_grad(dy, a, w, dA=want[0], dW=want[1], dbias=want[2])
        assert [g is not None for g in got] == want and torch.equal(got[i], full[i])
    nan = [torch.full_like(t, float("nan")) for t in (w, b)]
    da, dw, db = lib.ep_matmul_bias_act_grad(dy[:0], a[:0], w, dW=nan[0], dbias=nan[1])
    assert da.shape == (0, 24) and not dw.any() and not db.any()
    da, dw, db = lib.ep_matmul_bias_act_grad(dy[:, :0].contiguous(), a, w[:0], dA=torch.full_like(a, float("nan")), dbias=True)
    assert not da.any() and dw.shape == (0, 24) and db.shape == (0,)


# dW's sums run over M, dA's over N: few tiles of long sums beside many of short ones
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("mnk", [(16384, 384, 384), (8200, 768, 768), (10000, 520, 264), (600, 9000, 640), (9001, 301, 299),
                                 (4096, 4096, 256)], ids=str)
def test_grad_long_sums(lib, mnk, dtype):
    backward(lib, *mnk, dtype)


@pytest.mark.parametrize("mnk", [(768, 768, 4096), (300, 301, 9992), (1034, 640, 2504)], ids=str)
def test_long_sums(lib, mnk):
    forward(lib, *mnk, "f16", "silu")


@pytest.mark.parametrize("act", ["none", "quick_gelu"])
@pytest.mark.parametrize("mnk", [(16384, 768, 768), (2048, 2048, 1024), (600, 9000, 640)], ids=str)
def test_grad_many_calls(lib, mnk, act):
    """Calls queued one behind another, from a slow and from a fast host, and replayed: the first's bits."""
    m, n, k = mnk
    a, w, b, r = cuda(*product_inputs(m, n, k, "bf16", 9))
    args = r, a, w, (r if act != "none" else None), act_code(lib, act)
    first = lib.ep_matmul_bias_act_grad(*args)[:2]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for pause in (0, 20e-6, 60e-6):
            for _ in range(100):
                out = lib.ep_matmul_bias_act_grad(*args)[:2]
                t = time.perf_counter()
                while time.perf_counter() - t < pause:
                    pass
            assert all(torch.equal(x, y) for x, y in zip(out, first))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs = [lib.ep_matmul_bias_act_grad(*args)[:2] for _ in range(4)]
        for _ in range(20):
            g.replay()
        s.synchronize()
        for out in outs:
            assert all(torch.equal(x, y) for x, y in zip(out, first))
    assert lib.ep_pipeline_timeouts() == 0


@pytest.mark.parametrize("mnk,mx8", [((2048, 2048, 1024), True), ((1300, 1001, 771), True), ((1300, 1001, 771), False),
                                     ((16, 4096, 4096), True)], ids=str)
def test_many_calls(lib, mnk, mx8):
    """The same of the product, with the copies and arranged scales in front of it."""
    a, w, b, r = cuda(*product_inputs(*mnk, "f16", 10))
    kw = {}
    if mx8:
        (a, sa), (w, sw) = lib.ep_quantize_mx8(a), lib.ep_quantize_mx8(w)
        kw = dict(A_scales=sa, W_scales=sw, dtype=r.dtype)

    def call():
        return lib.ep_matmul_bias_act(a, w, b, r, lib.EP_ACT_SILU, Z=E4M3, **kw)
    first = [x.view(torch.uint8) for x in call()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for pause in (0, 20e-6, 60e-6):
            for _ in range(200):
                out = call()
                t = time.perf_counter()
                while time.perf_counter() - t < pause:
                    pass
            assert all(torch.equal(x.view(torch.uint8), y) for x, y in zip(out, first))
    assert lib.ep_pipeline_timeouts() == 0
