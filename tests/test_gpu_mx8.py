"""MX8 rows and the RMS norm with its gradient against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import products as op
from tests._helpers import U32
from tests._products import (DT, assert_mx8, assert_within, at_offset, cuda, f64, mx8_f64, scale_bytes)

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (3, 7), (5, 31), (4, 32), (2, 33), (9, 64), (3, 100), (1, 4096), (7, 8), (257, 72), (2, 3, 200),
          (5, 1001), (3, 4100), (2, 8192), (2, 16384), (2, 16392), (3, 20001), (1030, 24)]


def rows(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize_is_exact(lib, shape, dtype):
    x = rows(shape, dtype, 1, 3.0)
    x.view(-1)[:: 7] *= 64
    q, s = lib.ep_quantize_mx8(x.cuda())
    n = shape[-1]
    wq, wb = op.mx8_quantize(f64(x).reshape(-1, n))
    assert s.shape == tuple(shape[:-1]) + (-(-n // 32),)
    np.testing.assert_array_equal(scale_bytes(s).reshape(wb.shape), wb)
    np.testing.assert_array_equal(q.float().double().cpu().numpy().reshape(wq.shape), wq)
    y = lib.ep_dequantize_mx8(q, s, DT[dtype])
    np.testing.assert_array_equal(f64(y).reshape(wq.shape), op.mx8_values(wq, wb))


@pytest.mark.parametrize("width", [32, 33])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_edges(lib, width, dtype):
    """Zeros, the smallest and largest numbers, every power of two and the values beside the scales' borders."""
    fi = torch.finfo(DT[dtype])
    vals = [0.0, -0.0, fi.tiny, fi.smallest_normal, fi.max, -fi.max, 448.0, 449.0, 464.0, 480.0, 2.0 ** -120, 2.0 ** -126]
    vals += [2.0 ** e for e in range(-126, 128, 3)] + [1.75 * 2.0 ** e for e in range(-120, 127, 5)]
    x = torch.zeros(len(vals), width, dtype=torch.float64)
    for i, v in enumerate(vals):
        x[i, i % width] = v
        x[i, (i + 3) % width] = -v * 0.3
    x = x.to(DT[dtype])
    q, s = lib.ep_quantize_mx8(x.cuda())
    wq, wb = op.mx8_quantize(f64(x))
    np.testing.assert_array_equal(scale_bytes(s), wb)
    np.testing.assert_array_equal(q.float().double().cpu().numpy(), wq)
    with np.errstate(over="ignore"):  # the largest float32 rounds up to 2^128, which float32 lacks
        want = op.mx8_values(wq, wb).astype(np.float32)
    np.testing.assert_array_equal(lib.ep_dequantize_mx8(q, s, torch.float32).cpu().numpy(), want)


@pytest.mark.parametrize("width", [64, 71])
def test_nan_and_infinity(lib, width):
    x = torch.randn(4, width, dtype=torch.float32, generator=torch.Generator().manual_seed(2))
    x[0, 3], x[1, 40], x[2, 40], x[3, :] = float("nan"), float("inf"), float("-inf"), float("nan")
    q, s = lib.ep_quantize_mx8(x.cuda())
    got, b = mx8_f64(q, s), scale_bytes(s)
    assert np.isnan(got[0, 3]) and np.isfinite(np.delete(got[0], 3)).all()
    for r in (1, 2):
        assert b[r, 1] == 255 and np.isnan(got[r, 32:64]).all() and np.isfinite(got[r, :32]).all()
    assert np.isnan(got[3]).all()
    back = f64(lib.ep_dequantize_mx8(q, s, torch.float32))
    np.testing.assert_array_equal(np.isnan(back), np.isnan(got))


def test_dequantize_every_byte(lib):
    """All E4M3 bytes under all scales, against torch's conversions of either."""
    q = torch.arange(256, dtype=torch.uint8).repeat(256, 1).view(torch.float8_e4m3fn)
    s = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 8).view(torch.float8_e8m0fnu)
    y = lib.ep_dequantize_mx8(q.cuda(), s.cuda(), torch.float32).cpu()
    b = torch.arange(256, dtype=torch.float64).view(256, 1)
    want = q.float().double() * torch.where(b == 255, float("nan"), torch.exp2(b - 127))
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(y[ok].double(), want[ok].float().double())


@pytest.mark.parametrize("off", [1, 4])
def test_quantize_alignments(lib, off):
    x = cuda(rows((6, 96), "f16", 3))
    q0, s0 = lib.ep_quantize_mx8(x)
    buf = torch.zeros(6 * 96 + 16, dtype=torch.uint8, device="cuda")
    qv = buf[off:off + 6 * 96].view(6, 96).view(torch.float8_e4m3fn)
    q1, s1 = lib.ep_quantize_mx8(at_offset(x, off), Q=qv, scales=torch.empty_like(s0))
    assert torch.equal(q0.view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s0.view(torch.uint8), s1.view(torch.uint8))
    y0, y1 = lib.ep_dequantize_mx8(q0, s0, torch.float16), lib.ep_dequantize_mx8(qv, s1, torch.float16)
    assert torch.equal(y0, y1)
    assert not buf[:off].any() and not buf[off + 6 * 96:].any()


def norm_case(lib, shape, dtype, seed, skip=True, bias=True, eps=1e-6, off=0):
    h = shape[-1]
    x, sk = rows(shape, dtype, seed), rows(shape, dtype, seed + 1, 0.5) if skip else None
    g, b = (rows((h,), dtype, seed + 2) * 0.2 + 1).to(DT[dtype]), rows((h,), dtype, seed + 3, 0.1) if bias else None
    dev = [at_offset(t, off) if off else t for t in cuda(x, sk, g, b)]
    q, s, su, inv = lib.ep_skip_rms_norm_mx8(*dev, epsilon=eps, input_skip_bias_sum=True, inv_std_dev=True)
    o = op.rms_norm(*(None if t is None else f64(t).reshape(-1, h) if t.dim() > 1 else f64(t) for t in (x, sk, g, b)), eps)
    # s: two roundings of its terms; inv: as GroupNorm's, 64 u; three more roundings
    sd = 2 * U32 * o["terms"]
    want = x.float() if sk is None else x.float() + sk.float()
    if b is not None:
        want = want + b.float()
    assert torch.equal(su.cpu(), want.to(DT[dtype]))
    inv_rel = 64 * U32 + 2 * (sd * np.abs(o["s"])).mean(axis=1, keepdims=True) * o["inv"] ** 2
    assert_within(inv.reshape(-1, 1), o["inv"], inv_rel * o["inv"], "rms inv")
    delta = np.abs(o["y"]) * (inv_rel + 4 * U32) + sd * o["inv"] * np.abs(f64(g))
    assert_mx8(q, s, o["y"], delta, "rms q")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm(lib, shape, dtype):
    norm_case(lib, shape, dtype, 11)


@pytest.mark.parametrize("skip,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("shape", [(5, 768), (4, 77)], ids=str)
def test_norm_without(lib, shape, skip, bias):
    norm_case(lib, shape, "bf16", 12, skip, bias)


@pytest.mark.parametrize("off", [1, 8])
def test_norm_alignments(lib, off):
    norm_case(lib, (7, 512), "f16", 13, off=off)


def test_norm_matches_the_simplified_form(lib):
    """The sum and the statistic are those of ep_skip_layer_norm_ex (simplified); the 8-bit rows stand for its output."""
    x, sk, g = cuda(rows((64, 1024), "bf16", 14), rows((64, 1024), "bf16", 15), rows((1024,), "bf16", 16, 0.1) + 1)
    y, su, _, inv = lib.ep_skip_layer_norm_ex(x, sk, g, epsilon=1e-6, simplified=True, input_skip_bias_sum=True,
                                              inv_std_dev=True)
    q, s, su8, inv8 = lib.ep_skip_rms_norm_mx8(x, sk, g, epsilon=1e-6, input_skip_bias_sum=True, inv_std_dev=True)
    assert torch.equal(su, su8)
    assert torch.allclose(inv.view(-1), inv8.view(-1), rtol=128 * U32, atol=0)
    v = lib.ep_dequantize_mx8(q, s, torch.float32)
    amax = y.float().abs().view(64, 32, 32).amax(2).repeat_interleave(32, 1)
    # half a step of E4M3 (2^-4 of the value, and 2^-10 / 448 of the group's maximum, with its scale rounded
    # up by at most 2) and y's own rounding to bf16
    assert ((v - y.float()).abs() <= y.float().abs() * (2.0 ** -4 + 2.0 ** -8) + amax * 2.0 ** -17).all()


def test_norm_in_place_sum(lib):
    x, sk, g = cuda(rows((33, 2048), "f16", 17), rows((33, 2048), "f16", 18), rows((2048,), "f16", 19))
    want = lib.ep_skip_rms_norm_mx8(x, sk, g, input_skip_bias_sum=True)
    for i in (0, 1):
        a, b = x.clone(), sk.clone()
        got = lib.ep_skip_rms_norm_mx8(a, b, g, input_skip_bias_sum=(a, b)[i])
        for u, v in zip(want[:3], got[:3]):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


GRAD_SHAPES = [(1, 1), (3, 7), (5, 32), (9, 64), (3, 100), (1, 4096), (700, 8), (257, 72), (2, 300, 200), (1200, 1001),
               (5, 4100), (40, 4096), (3, 8192), (3, 16384), (66, 16392), (35, 20001), (5000, 24), (2000, 3)]


def grad_case(lib, shape, dtype, seed, dsum=True, dbias=True, off=0):
    h = shape[-1]
    s, dy = rows(shape, dtype, seed), rows(shape, dtype, seed + 1)
    ds = rows(shape, dtype, seed + 2) if dsum else None
    g = (rows((h,), dtype, seed + 3) * 0.2 + 1).to(DT[dtype])
    inv = (1.0 / torch.sqrt((s.double() ** 2).mean(-1, keepdim=True) + 1e-6)).float()
    d = [at_offset(t, off) if off else t for t in cuda(dy, s, g, inv, ds)]
    dx, dg, db = lib.ep_skip_rms_norm_grad(*d[:4], dsum=d[4], dbias=True if dbias else None)
    o = op.rms_norm_grad(f64(dy).reshape(-1, h), f64(s).reshape(-1, h), f64(g), f64(inv).reshape(-1, 1),
                         None if ds is None else f64(ds).reshape(-1, h))
    # the row's mean is a sum of depth below 100, dX some ten roundings; the column sums' depth is below 100 too
    assert_within(dx, o["dX"], 64 * U32 * o["dX_scale"], "rms dX")
    assert_within(dg, o["dgamma"], 128 * U32 * o["dgamma_scale"], "rms dgamma")
    if dbias:
        assert_within(db, o["dbias"], 128 * U32 * o["dbias_scale"], "rms dbias")
    else:
        assert db is None


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", GRAD_SHAPES, ids=str)
def test_norm_grad(lib, shape, dtype):
    grad_case(lib, shape, dtype, 21)


@pytest.mark.parametrize("dsum,dbias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("shape", [(50, 768), (40, 77), (7, 16400)], ids=str)
def test_norm_grad_without(lib, shape, dsum, dbias):
    grad_case(lib, shape, "bf16", 22, dsum, dbias)


@pytest.mark.parametrize("off", [1, 8])
def test_norm_grad_alignments(lib, off):
    grad_case(lib, (70, 512), "f16", 23, off=off)


@pytest.mark.parametrize("shape", [(33, 2048), (33, 77), (9, 20001)], ids=str)
def test_norm_grad_in_place(lib, shape):
    h = shape[-1]
    dy, s, ds = cuda(rows(shape, "f16", 24), rows(shape, "f16", 25), rows(shape, "f16", 26))
    g, inv = cuda(rows((h,), "f16", 27), torch.ones(shape[0], 1))
    want = lib.ep_skip_rms_norm_grad(dy, s, g, inv, dsum=ds, dbias=True)
    for i in range(3):
        c = [dy.clone(), s.clone(), ds.clone()]
        got = lib.ep_skip_rms_norm_grad(c[0], c[1], g, inv, dsum=c[2], dX=c[i], dbias=True)
        for u, v in zip(want, got):
            assert torch.equal(u, v)


# rows that start on no 16-byte boundary: element by element below 8 million elements or 96 a row, else in
# fragments that are cut at both ends (a row's phase repeats every 8 rows): rows of several slots a block, of whole
# blocks, and (16378 on) too long for them
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 65), (9, 65), (8, 68), (300, 127), (3000, 66), (77, 132), (601, 1003), (17, 8191),
                                   (88500, 95), (88000, 97), (84000, 100), (68000, 127),
                                   (26000, 325), (8500, 1003), (3400, 2525), (2100, 4100), (1700, 5034), (1050, 8191),
                                   (520, 16377), (520, 16378)], ids=str)
def test_norm_grad_odd_rows(lib, shape, dtype):
    grad_case(lib, shape, dtype, 31)
    if dtype == "f16":
        grad_case(lib, shape, dtype, 32, dsum=False, dbias=False)


@pytest.mark.parametrize("shape", [(9, 65), (68000, 127), (1700, 5034)], ids=str)
def test_norm_grad_odd_rows_ends(lib, shape):
    """dX over dY in the middle of a larger tensor: what lies around it stays, and NaN there is not taken in."""
    h = shape[-1]
    g = torch.Generator().manual_seed(33)
    s, ds, dy = (torch.randn(shape, generator=g).half().cuda() for _ in range(3))
    gamma, inv = torch.ones(h, dtype=torch.float16, device="cuda"), torch.ones(shape[0], 1, device="cuda")
    want = lib.ep_skip_rms_norm_grad(dy, s, gamma, inv, dsum=ds, dbias=True)
    n = dy.numel()
    bufs = [torch.full((n + 32,), float("nan"), dtype=torch.float16, device="cuda") for _ in range(3)]
    ins = [b[16:16 + n].view(shape) for b in bufs]
    for t, x in zip(ins, (dy, s, ds)):
        t.copy_(x)
    got = lib.ep_skip_rms_norm_grad(ins[0], ins[1], gamma, inv, dsum=ins[2], dX=ins[0], dbias=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for b in bufs:
        assert b[:16].isnan().all() and b[16 + n:].isnan().all()
