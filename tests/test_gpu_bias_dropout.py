"""BiasDropout and its gradient (through the C ABI) against the float64 oracle;
the mask is compared element by element."""
import numpy as np
import pytest
import torch

from oracle import training as tr
from tests._helpers import U32, Guarded, assert_bit_exact, offset_copy, to_np64
from tests._training import assert_within, dropout_inputs

pytestmark = pytest.mark.gpu

SEED, OFFSET = 0x1234567_89ABCDEF, 0xFEDCBA98_00000003

SHAPES = [(1,), (3,), (4,), (7,), (1, 1), (5, 1), (3, 2, 5), (2, 3, 8), (1, 8192), (9, 771), (33, 64), (2, 17, 189),
          (700, 24), (2, 3, 4, 40), (13, 4104), (3, 2055), (1, 100003), (4099, 3), (2, 5000, 16)]


def run(lib, d, ratio, offsets=None, seed=SEED, offset=OFFSET, alias=None):
    offsets = offsets or {}
    dev = {k: None if v is None else (offset_copy(v, offsets[k])[1] if k in offsets else v.cuda())
           for k, v in d.items()}
    y = Guarded(d["X"].shape, d["X"].dtype, offset_bytes=offsets.get("Y", 0))
    if alias is not None:
        y.tensor.copy_(dev[alias])
        dev[alias] = y.tensor
    lib.ep_bias_dropout(dev["X"], ratio, seed, offset, bias=dev["bias"], residual=dev["residual"], Y=y.tensor)
    torch.cuda.synchronize()
    y.check()
    return y.tensor.cpu()


def check(y, d, ratio, seed=SEED, offset=OFFSET):
    o = tr.bias_dropout(d["X"], ratio, seed, offset, d["bias"], d["residual"])
    assert_within(y, o["Y"], U32 * (3 * np.abs(o["kept"]) + np.abs(o["Y"])), "dropout")
    return o


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_bias_dropout_shapes(lib, dtype, shape):
    k = sum(shape)
    d = dropout_inputs(shape, dtype, k, bias=k % 3 != 0, residual=k % 2 == 0)
    check(run(lib, d, 0.3), d, 0.3)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("ratio", [0.0, 0.1, 0.5, 0.999, 1.0 - 2.0 ** -34])
def test_bias_dropout_mask_is_the_oracles(lib, dtype, ratio):
    d = dropout_inputs((64, 513), dtype, 3, bias=False, residual=False)
    y = run(lib, d, ratio)
    o = check(y, d, ratio)
    if ratio < 0.99:   # kept values stay finite and nonzero in every type
        assert np.array_equal(to_np64(y) != 0, o["keep"])


@pytest.mark.parametrize("dtype,offs", [
    ("f16", {"X": 2}), ("f16", {"Y": 2}), ("f16", {"bias": 6}), ("f32", {"residual": 4}), ("bf16", {"X": 8, "Y": 8}),
    ("f32", {"X": 8, "Y": 8, "residual": 8, "bias": 8})])
def test_bias_dropout_alignment(lib, dtype, offs):
    d = dropout_inputs((3, 9, 64), dtype, 1)
    check(run(lib, d, 0.4, offs), d, 0.4)


@pytest.mark.parametrize("alias", ["X", "residual"])
@pytest.mark.parametrize("shape", [(33, 64), (2, 17, 189)])
def test_bias_dropout_in_place(lib, alias, shape):
    d = dropout_inputs(shape, "bf16", 5)
    assert_bit_exact(run(lib, d, 0.25), run(lib, d, 0.25, alias=alias))


def test_bias_dropout_same_mask_for_every_type_and_alignment(lib):
    masks = []
    for dtype, offs in (("f32", None), ("f16", None), ("bf16", {"X": 2}), ("f16", {"Y": 6})):
        d = dropout_inputs((31, 77), dtype, 9, bias=False, residual=False)
        masks.append(run(lib, d, 0.5, offs) != 0)
    assert all(torch.equal(m, masks[0]) for m in masks)


def test_bias_dropout_dropped_elements_ignore_what_is_there(lib):
    d = dropout_inputs((40, 96), "f32", 13)
    keep = torch.from_numpy(tr.dropout_keep(40 * 96, 0.5, SEED, OFFSET)).view(40, 96)
    want = run(lib, d, 0.5)
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = torch.where(keep, d["X"], torch.full_like(d["X"], bad))
        assert torch.equal(run(lib, dict(d, X=x), 0.5), want)
    x = d["X"].clone()
    x[keep] = float("inf")
    y = run(lib, dict(d, X=x), 0.5)
    assert torch.isinf(y[keep]).all() and torch.isfinite(y[~keep]).all()


def test_bias_dropout_counter_beyond_32_bits_of_offset(lib):
    d = dropout_inputs((16, 128), "f32", 17, bias=False, residual=False)
    for seed, offset in ((0, 0), (1 << 32, 0), (0, 1 << 32), ((1 << 64) - 1, (1 << 64) - 1)):
        check(run(lib, d, 0.5, seed=seed, offset=offset), d, 0.5, seed, offset)


def test_bias_dropout_offset_from_device_memory(lib):
    d = dropout_inputs((16, 130), "f16", 19, residual=False)
    x, b = d["X"].cuda(), d["bias"].cuda()
    step = torch.tensor([5], dtype=torch.int64, device="cuda")
    y = lib.ep_bias_dropout(x, 0.5, SEED, OFFSET, bias=b, offset_device=step)
    assert_bit_exact(y.cpu(), run(lib, d, 0.5, offset=OFFSET + 5))
    dx, db = lib.ep_bias_dropout_grad(x, 0.5, SEED, OFFSET, offset_device=step, dbias=True)
    want = lib.ep_bias_dropout_grad(x, 0.5, SEED, OFFSET + 5, dbias=True)
    assert torch.equal(dx, want[0]) and torch.equal(db, want[1])
    step.fill_(-1)   # 2^64 - 1: the sum wraps
    y = lib.ep_bias_dropout(x, 0.5, SEED, 7, bias=b, offset_device=step)
    assert_bit_exact(y.cpu(), run(lib, d, 0.5, offset=6))


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------

def gradient(lib, dy, ratio, offset_bytes=0, in_place=False, with_bias=True):
    src = offset_copy(dy, offset_bytes)[1] if offset_bytes else dy.cuda()
    dx = Guarded(dy.shape, dy.dtype, offset_bytes=offset_bytes)
    if in_place:
        dx.tensor.copy_(src)
        src = dx.tensor
    db = Guarded(dy.shape[-1:], dy.dtype)
    lib.ep_bias_dropout_grad(src, ratio, SEED, OFFSET, dX=dx.tensor, dbias=db.tensor if with_bias else None)
    torch.cuda.synchronize()
    dx.check()
    db.check()
    return dx.tensor.cpu(), db.tensor.cpu()


def check_gradient(dx, db, dy, ratio):
    o = tr.bias_dropout_grad(dy, ratio, SEED, OFFSET)
    assert_within(dx, o["dX"], 2 * U32 * np.abs(o["dX"]), "dropout dX")
    assert_within(db, o["dbias"], 64 * U32 * o["dbias_scale"], "dropout dbias")
    assert np.array_equal(to_np64(dx) != 0, o["keep"])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_bias_dropout_grad_shapes(lib, dtype, shape):
    dy = dropout_inputs(shape, dtype, sum(shape) + 1)["X"]
    dx, db = gradient(lib, dy, 0.3)
    check_gradient(dx, db, dy, 0.3)
    assert_bit_exact(gradient(lib, dy, 0.3, with_bias=False)[0], dx)


@pytest.mark.parametrize("dtype,offset", [("f32", 4), ("f16", 2), ("bf16", 8)])
@pytest.mark.parametrize("shape", [(33, 64), (2, 17, 189), (13, 4104)])
def test_bias_dropout_grad_alignment(lib, dtype, offset, shape):
    dy = dropout_inputs(shape, dtype, 27)["X"]
    dx, db = gradient(lib, dy, 0.5, offset)
    check_gradient(dx, db, dy, 0.5)


def test_bias_dropout_grad_in_place(lib):
    dy = dropout_inputs((300, 200), "f16", 29)["X"]
    for a, b in zip(gradient(lib, dy, 0.2), gradient(lib, dy, 0.2, in_place=True)):
        assert_bit_exact(a, b)


def test_bias_dropout_grad_sums_what_is_not_yet_rounded(lib):
    # 2^-9 of dx is lost by its rounding to bf16, always the same way: a sum of
    # the rounded values would be off by 2^-9 of dbias, four times its own spacing
    n = 4096
    dy = torch.full((n, 8), 1.0 + 2.0 ** -7, dtype=torch.bfloat16)
    dx, db = gradient(lib, dy, 0.3)
    check_gradient(dx, db, dy, 0.3)


def test_bias_dropout_grad_is_the_derivative(lib):
    # y is linear in x and bias: with residual 0 and float32 values whose
    # products are exact (ratio 1/2, small integers), differences are exact
    g = torch.Generator().manual_seed(31)
    x = torch.randint(-8, 9, (50, 36), generator=g).float().cuda()
    b = torch.randint(-8, 9, (36,), generator=g).float().cuda()
    w = torch.randint(-8, 9, (50, 36), generator=g).float().cuda()
    vx = torch.randint(-4, 5, (50, 36), generator=g).float().cuda()
    vb = torch.randint(-4, 5, (36,), generator=g).float().cuda()
    y0 = lib.ep_bias_dropout(x, 0.5, SEED, OFFSET, bias=b)
    y1 = lib.ep_bias_dropout(x + vx, 0.5, SEED, OFFSET, bias=b + vb)
    dx, db = lib.ep_bias_dropout_grad(w, 0.5, SEED, OFFSET, dbias=True)
    assert float(((y1 - y0) * w).sum()) == float((dx * vx).sum() + (db * vb).sum())


def test_bias_dropout_grad_repeats_bit_for_bit(lib):
    dy = dropout_inputs((5000, 96), "f32", 37)["X"].cuda()
    first = lib.ep_bias_dropout_grad(dy, 0.1, SEED, OFFSET, dbias=True)
    for _ in range(3):
        again = lib.ep_bias_dropout_grad(dy, 0.1, SEED, OFFSET, dbias=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_bias_dropout_empty_tensors(lib):
    x = torch.empty((0, 8), dtype=torch.float16, device="cuda")
    assert lib.ep_bias_dropout(x, 0.5, 1).shape == x.shape
    dx, db = lib.ep_bias_dropout_grad(x, 0.5, 1, dbias=True)
    assert dx.shape == x.shape and db.shape == (8,) and not db.any()


def test_bias_dropout_workspace(lib):
    dy = dropout_inputs((3000, 72), "f16", 41)["X"].cuda()
    want = lib.ep_bias_dropout_grad(dy, 0.5, SEED, OFFSET, dbias=True)
    need = lib.ep_bias_dropout_grad_workspace_size(torch.float16, (3000, 72))
    assert need > 0
    ws = torch.full((need + 32,), 0xFF, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = lib.ep_bias_dropout_grad(dy, 0.5, SEED, OFFSET, dbias=True, workspace=ws[:need], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert bool((ws[need:] == 0xFF).all())
    with pytest.raises(lib.EpError) as e:
        lib.ep_bias_dropout_grad(dy, 0.5, SEED, OFFSET, dbias=True, workspace=ws[:need - 16])
    assert e.value.status == lib.EP_ERR_WORKSPACE
