"""What fixes the order of the sums: the shape alone for the product and its gradient, the shape and the
operands' alignment to 16 bytes for the RMS norm and its gradient."""
import os

import pytest
import torch

from tests._products import at_offset

E4M3 = torch.float8_e4m3fn


def draws(*shapes, dtype):
    g = torch.Generator(device="cuda").manual_seed(61)
    return [torch.randn(*s, device="cuda", generator=g).to(dtype) for s in shapes]


def bits(out):
    return [t.view(torch.uint8) if t.element_size() == 1 else t for t in out if t is not None]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(5, 72, 96), (130, 264, 72), (1040, 2568, 64), (300, 301, 1001)])
@pytest.mark.parametrize("off", [1, 3, 8])
def test_product_at_any_address(lib, m, n, k, off):
    a, w, b, r = draws((m, k), (n, k), (n,), (m, n), dtype=torch.float16)
    z = r * 2
    (qa, sa), (qw, sw) = lib.ep_quantize_mx8(a), lib.ep_quantize_mx8(w)

    def run(*t):
        a, w, b, r, z, qa, sa, qw, sw = t
        return (lib.ep_matmul_bias_act(a, w, b, r, lib.EP_ACT_GELU, Z=E4M3)
                + lib.ep_matmul_bias_act(qa, qw, b, r, lib.EP_ACT_SILU, A_scales=sa, W_scales=sw, Z=True)
                + lib.ep_matmul_bias_act_grad(r, a, w, z, lib.EP_ACT_QUICK_GELU, dbias=True))
    ins = (a, w, b, r, z, qa, sa, qw, sw)
    for x, y in zip(bits(run(*ins)), bits(run(*(at_offset(t, off) for t in ins)))):
        assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,h", [(9, 40), (33, 768), (70, 4100), (5, 20001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_norm_at_another_address_of_the_same_alignment(lib, rows, h, dtype):
    x, sk, dy, ds = draws(*[(rows, h)] * 4, dtype=dtype)
    g, = draws((h,), dtype=dtype)
    step = 16 // x.element_size()

    def run(off):
        v = [at_offset(t, off) for t in (x, sk, g, dy, ds)]
        q, s, su, inv = lib.ep_skip_rms_norm_mx8(*v[:3], input_skip_bias_sum=True, inv_std_dev=True)
        return (q, s, su, inv) + lib.ep_skip_rms_norm_grad(v[3], at_offset(su, off), v[2], inv, dsum=v[4], dbias=True)
    for off in (0, 1):
        for a, b in zip(bits(run(off)), bits(run(off + step))):
            assert torch.equal(a, b)


def test_the_header_says_so():
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ep.h"), encoding="utf-8") as f:
        text = " ".join(f.read().replace(" * ", " ").split())
    norm = text[text.index("RMS norm with the residual"):text.index("Matrix product with bias")]
    assert norm.count("fixed by the shape and by which operands start on 16-byte boundaries") == 2
    assert "fixed order" not in norm
