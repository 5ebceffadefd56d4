"""Host-side contract checks of MX8 rows, the RMS norm and the matrix product, run in
a subprocess with no visible CUDA device (CUDA_VISIBLE_DEVICES=""), as
abi_training_cases.py: the addresses are placeholders that nothing reads, and a case
that passes the checks ends in the device query (EP_ERR_CUDA)."""
import ctypes
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

F32, F16, BF16, F64 = 0, 1, 2, 7
OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4
P = [0x700000000000 + i * (1 << 42) for i in range(14)]
BIG = 1 << 41   # workspace bytes
MOST = (1 << 31) - 512


def shp(*d):
    return None if d == (None,) else (ctypes.c_int64 * max(1, len(d)))(*d)


def quant(lib, t=F16, x=P[0], shape=(3, 40), rank=None, q=P[1], s=P[2]):
    return lib.ep_quantize_mx8(t, x, None if shape is None else shp(*shape), len(shape or ()) if rank is None else rank,
                               q, s, None)


def dequant(lib, t=F16, q=P[0], s=P[1], shape=(3, 40), rank=None, y=P[2]):
    return lib.ep_dequantize_mx8(t, q, s, None if shape is None else shp(*shape),
                                 len(shape or ()) if rank is None else rank, y, None)


def norm(lib, t=F16, x=P[0], shape=(3, 40), skip=P[1], gamma=P[2], bias=P[3], eps=1e-6, q=P[4], s=P[5], total=P[6], inv=P[7]):
    return lib.ep_skip_rms_norm_mx8(t, x, None if shape is None else shp(*shape), len(shape or ()), skip, gamma, bias, eps,
                                    q, s, total, inv, None)


def normg(lib, t=F16, dy=P[0], s=P[1], shape=(3, 40), gamma=P[2], inv=P[3], dsum=P[4], dx=P[5], dg=P[6], db=P[7], ws=P[8],
          wsb=BIG):
    return lib.ep_skip_rms_norm_grad(t, dy, s, None if shape is None else shp(*shape), len(shape or ()), gamma, inv, dsum,
                                     dx, dg, db, ws, wsb, None)


def mm(lib, t=BF16, a=P[0], w=P[1], m=6, n=40, k=24, bias=P[2], res=P[3], act=0, alpha=1.7, y=P[4], z=P[5], zs=None, ws=P[7],
       wsb=BIG):
    return lib.ep_matmul_bias_act(t, a, w, m, n, k, bias, res, act, alpha, y, z, zs, ws, wsb, None)


def mm8(lib, t=BF16, a=P[0], sa=P[8], w=P[1], sw=P[9], m=6, n=40, k=32, bias=P[2], res=P[3], act=0, alpha=1.7, y=P[4], z=P[5],
        zs=P[6], ws=P[7], wsb=BIG):
    return lib.ep_matmul_bias_act_mx8(t, a, sa, w, sw, m, n, k, bias, res, act, alpha, y, z, zs, ws, wsb, None)


def mmg(lib, t=BF16, dy=P[0], a=P[1], sa=None, w=P[2], z=P[3], zs=None, m=6, n=40, k=24, act=1, alpha=1.7, da=P[4], dw=P[5],
        db=P[6], ws=P[7], wsb=BIG):
    return lib.ep_matmul_bias_act_grad(t, dy, a, sa, w, z, zs, m, n, k, act, alpha, da, dw, db, ws, wsb, None)


def cases(lib):
    nan, inf = float("nan"), float("inf")
    out = [
        ("quant ok", quant(lib), CUDA), ("quant f32 ok", quant(lib, t=F32), CUDA), ("quant 1-d ok", quant(lib, shape=(7,)), CUDA),
        ("quant dtype", quant(lib, t=F64), UNSUPPORTED), ("quant NULL shape", quant(lib, shape=None, rank=2), INVALID),
        ("quant rank 0", quant(lib, shape=()), INVALID), ("quant rank 17", quant(lib, shape=(1,) * 17), UNSUPPORTED),
        ("quant negative", quant(lib, shape=(-1, 8)), INVALID), ("quant overflow", quant(lib, shape=(1 << 40, 1 << 40)), INVALID),
        ("quant H", quant(lib, shape=(1, MOST + 1)), UNSUPPORTED), ("quant rows", quant(lib, shape=((1 << 33) + 1, 1)), UNSUPPORTED),
        ("quant empty", quant(lib, shape=(0, 8), x=None, q=None, s=None), OK),
        ("quant H = 0", quant(lib, shape=(8, 0), x=None, q=None, s=None), OK),
        ("quant NULL x", quant(lib, x=None), INVALID), ("quant NULL q", quant(lib, q=None), INVALID),
        ("quant NULL scales", quant(lib, s=None), INVALID), ("quant misaligned", quant(lib, x=P[0] + 1), INVALID),
        ("quant q odd ok", quant(lib, q=P[1] + 3, s=P[2] + 1), CUDA),
        ("quant in place", quant(lib, q=P[0]), INVALID), ("quant overlap", quant(lib, s=P[1] + 60), INVALID),
        ("quant scales behind ok", quant(lib, s=P[1] + 120), CUDA),
        ("dequant ok", dequant(lib), CUDA), ("dequant dtype", dequant(lib, t=F64), UNSUPPORTED),
        ("dequant NULL", dequant(lib, q=None), INVALID), ("dequant NULL scales", dequant(lib, s=None), INVALID),
        ("dequant NULL y", dequant(lib, y=None), INVALID), ("dequant misaligned", dequant(lib, y=P[2] + 1), INVALID),
        ("dequant overlap", dequant(lib, y=P[1] - 8), INVALID), ("dequant empty", dequant(lib, shape=(0, 3), q=None), OK),
        ("norm ok", norm(lib), CUDA), ("norm f32 ok", norm(lib, t=F32), CUDA),
        ("norm without ok", norm(lib, skip=None, bias=None, total=None, inv=None), CUDA),
        ("norm dtype", norm(lib, t=F64), UNSUPPORTED), ("norm NULL shape", norm(lib, shape=None), INVALID),
        ("norm H = 0", norm(lib, shape=(3, 0)), INVALID), ("norm no rows", norm(lib, shape=(0, 8), x=None), OK),
        ("norm eps", norm(lib, eps=-1.0), INVALID), ("norm NaN eps", norm(lib, eps=nan), INVALID),
        ("norm eps 0 ok", norm(lib, eps=0.0), CUDA),
        ("norm NULL x", norm(lib, x=None), INVALID), ("norm NULL gamma", norm(lib, gamma=None), INVALID),
        ("norm NULL q", norm(lib, q=None), INVALID), ("norm NULL scales", norm(lib, s=None), INVALID),
        ("norm misaligned", norm(lib, gamma=P[2] + 1), INVALID), ("norm misaligned inv", norm(lib, inv=P[7] + 2), INVALID),
        ("norm sum in place ok", norm(lib, total=P[0]), CUDA), ("norm sum is skip ok", norm(lib, total=P[1]), CUDA),
        ("norm sum overlaps", norm(lib, total=P[0] + 2), INVALID), ("norm sum is bias", norm(lib, total=P[3]), INVALID),
        ("norm q is x", norm(lib, q=P[0]), INVALID), ("norm scales in q", norm(lib, s=P[4] + 1), INVALID),
        ("norm inv in gamma", norm(lib, inv=P[2] + 4), INVALID), ("norm inv in sum", norm(lib, inv=P[6]), INVALID),
        ("normg ok", normg(lib), CUDA), ("normg without ok", normg(lib, dsum=None, dg=None, db=None), CUDA),
        ("normg dtype", normg(lib, t=F64), UNSUPPORTED), ("normg H = 0", normg(lib, shape=(3, 0)), INVALID),
        ("normg NULL dy", normg(lib, dy=None), INVALID), ("normg NULL s", normg(lib, s=None), INVALID),
        ("normg NULL gamma", normg(lib, gamma=None), INVALID), ("normg NULL inv", normg(lib, inv=None), INVALID),
        ("normg NULL dx", normg(lib, dx=None), INVALID), ("normg misaligned", normg(lib, dg=P[6] + 1), INVALID),
        ("normg misaligned inv", normg(lib, inv=P[3] + 2), INVALID),
        ("normg dx = dy ok", normg(lib, dx=P[0]), CUDA), ("normg dx = s ok", normg(lib, dx=P[1]), CUDA),
        ("normg dx = dsum ok", normg(lib, dx=P[4]), CUDA), ("normg dx overlaps", normg(lib, dx=P[0] + 2), INVALID),
        ("normg dg is gamma", normg(lib, dg=P[2]), INVALID), ("normg dg = db", normg(lib, db=P[6]), INVALID),
        ("normg dg in dx", normg(lib, dg=P[5] + 8), INVALID),
        ("normg no workspace", normg(lib, ws=None), WORKSPACE), ("normg small", normg(lib, wsb=16), WORKSPACE),
        ("normg ws misaligned", normg(lib, ws=P[8] + 8), WORKSPACE), ("normg ws overlaps", normg(lib, ws=P[5]), WORKSPACE),
        ("mm ok", mm(lib), CUDA), ("mm f16 ok", mm(lib, t=F16), CUDA), ("mm f32", mm(lib, t=F32), UNSUPPORTED),
        ("mm f64", mm(lib, t=F64), UNSUPPORTED), ("mm without ok", mm(lib, bias=None, res=None, z=None), CUDA),
        ("mm negative m", mm(lib, m=-1), INVALID), ("mm negative n", mm(lib, n=-1), INVALID), ("mm negative k", mm(lib, k=-1), INVALID),
        ("mm m", mm(lib, m=MOST + 1, n=1, k=1), UNSUPPORTED), ("mm n", mm(lib, n=MOST + 1, m=1, k=1), UNSUPPORTED),
        ("mm k", mm(lib, k=MOST + 1, m=1, n=1), UNSUPPORTED), ("mm large", mm(lib, m=1 << 21, n=1 << 20, k=1), UNSUPPORTED),
        ("mm no rows", mm(lib, m=0, a=None, w=None, y=None), OK), ("mm no columns", mm(lib, n=0, a=None, w=None, y=None), OK),
        ("mm no depth ok", mm(lib, k=0, a=None, w=None), CUDA),
        ("mm NULL a", mm(lib, a=None), INVALID), ("mm NULL w", mm(lib, w=None), INVALID), ("mm NULL y", mm(lib, y=None), INVALID),
        ("mm act 6", mm(lib, act=6), INVALID), ("mm act -1", mm(lib, act=-1), INVALID), ("mm alpha", mm(lib, alpha=nan), INVALID),
        ("mm alpha inf", mm(lib, alpha=inf), INVALID), ("mm odd a", mm(lib, a=P[0] + 1), INVALID),
        ("mm odd bias", mm(lib, bias=P[2] + 1), INVALID), ("mm odd z", mm(lib, z=P[5] + 1), INVALID),
        ("mm odd z8 ok", mm(lib, z=P[5] + 1, zs=P[6] + 1), CUDA), ("mm scales without z", mm(lib, z=None, zs=P[6]), INVALID),
        ("mm y = res ok", mm(lib, y=P[3]), CUDA), ("mm y overlaps res", mm(lib, y=P[3] + 2), INVALID),
        ("mm y in a", mm(lib, y=P[0] + 8), INVALID), ("mm y is w", mm(lib, y=P[1]), INVALID), ("mm y is bias", mm(lib, y=P[2]), INVALID),
        ("mm z = res", mm(lib, z=P[3]), INVALID), ("mm z in y", mm(lib, z=P[4] + 8), INVALID),
        ("mm unaligned no workspace", mm(lib, a=P[0] + 2, ws=None), WORKSPACE),
        ("mm odd k no workspace", mm(lib, k=23, ws=None), WORKSPACE), ("mm no workspace needed ok", mm(lib, ws=None, wsb=0), CUDA),
        ("mm odd k small", mm(lib, k=23, wsb=64), WORKSPACE), ("mm odd k ws in y", mm(lib, k=23, ws=P[4]), WORKSPACE),
        ("mm8 ok", mm8(lib), CUDA), ("mm8 f32", mm8(lib, t=F32), UNSUPPORTED), ("mm8 NULL scales", mm8(lib, sa=None), INVALID),
        ("mm8 NULL w scales", mm8(lib, sw=None), INVALID), ("mm8 byte addresses ok", mm8(lib, a=P[0] + 1, sa=P[8] + 3), CUDA),
        ("mm8 z scales in z", mm8(lib, zs=P[5] + 9), INVALID), ("mm8 z scales in w's", mm8(lib, zs=P[9]), INVALID),
        ("mm8 large no workspace", mm8(lib, m=8192, n=8192, k=4096, ws=None), WORKSPACE),
        ("mm8 no depth ok", mm8(lib, k=0, a=None, w=None, sa=None, sw=None), CUDA),
        ("mmg ok", mmg(lib), CUDA), ("mmg f32", mmg(lib, t=F32), UNSUPPORTED), ("mmg 8-bit ok", mmg(lib, sa=P[8], zs=P[9]), CUDA),
        ("mmg no z", mmg(lib, z=None), INVALID), ("mmg no z needed ok", mmg(lib, act=0, z=None), CUDA),
        ("mmg no dy", mmg(lib, dy=None), INVALID), ("mmg dw without a", mmg(lib, a=None), INVALID),
        ("mmg da without w", mmg(lib, w=None), INVALID), ("mmg a not needed ok", mmg(lib, a=None, dw=None), CUDA),
        ("mmg w not needed ok", mmg(lib, w=None, da=None), CUDA), ("mmg act", mmg(lib, act=9), INVALID),
        ("mmg alpha", mmg(lib, alpha=inf), INVALID), ("mmg negative", mmg(lib, k=-2), INVALID),
        ("mmg misaligned", mmg(lib, da=P[4] + 1), INVALID), ("mmg byte a ok", mmg(lib, a=P[1] + 1, sa=P[8] + 1), CUDA),
        ("mmg byte a without scales", mmg(lib, a=P[1] + 1), INVALID),
        ("mmg da is dy", mmg(lib, da=P[0]), INVALID), ("mmg da in a", mmg(lib, da=P[1]), INVALID), ("mmg dw is w", mmg(lib, dw=P[2]), INVALID),
        ("mmg dw = da", mmg(lib, dw=P[4]), INVALID), ("mmg db in z", mmg(lib, db=P[3]), INVALID),
        ("mmg no workspace", mmg(lib, ws=None), WORKSPACE), ("mmg small", mmg(lib, wsb=64), WORKSPACE),
        ("mmg ws misaligned", mmg(lib, ws=P[7] + 8), WORKSPACE), ("mmg ws overlaps", mmg(lib, ws=P[6]), WORKSPACE),
        ("mmg no columns ok", mmg(lib, n=0, dy=None, z=None, w=None, dw=None, db=None), CUDA),
    ]
    return out


def sizes(lib):
    """(name, holds) of the workspace sizes."""
    f, g, r = (lib.ep_matmul_bias_act_workspace_size, lib.ep_matmul_bias_act_grad_workspace_size,
               lib.ep_skip_rms_norm_grad_workspace_size)
    s = shp(16, 64)
    return [
        ("mm aligned", f(0, 16, 40, 64, 1) == 0), ("mm anywhere", f(0, 16, 40, 64, 0) >= (16 + 40) * 64 * 2),
        ("mm ragged", f(0, 16, 40, 63, 1) >= (16 + 40) * 64 * 2), ("mm rejected", f(0, -1, 40, 64, 0) == 0),
        ("mm too large", f(0, 1 << 32, 40, 64, 0) == 0), ("mm empty", f(0, 0, 40, 64, 0) == 0),
        ("mx8 few", f(1, 16, 40, 64, 1) == 0), ("mx8 ragged", f(1, 16, 40, 63, 1) >= (16 + 40) * 64),
        ("mx8 many arrange their scales", f(1, 8192, 8192, 4096, 1) >= (8192 + 8192) * 128),
        ("grad has dbias's sums", g(16, 40, 64, 0, 0, 1) >= 40 * 4), ("grad has dz", g(16, 40, 64, 1, 0, 1) >= 16 * 40 * 2),
        ("grad has A", g(16, 40, 64, 0, 1, 1) >= 16 * 64 * 2 + 40 * 4), ("grad rejected", g(16, 40, -1, 0, 0, 1) == 0),
        ("grad anywhere", g(16, 40, 64, 0, 0, 0) >= (16 * 40 + 16 * 64 + 40 * 64) * 2),
        ("norm grad", r(1, s, 2) >= 16 * 64 * 4 // 16), ("norm grad rejected", r(9, s, 2) == 0 and r(1, s, 0) == 0),
    ]


def main():
    from transformer_epilogue_gb300 import _binding
    lib = _binding.raw()
    got = cases(lib)
    bad = [(name, st, want) for name, st, want in got if st != want]
    bad += [(name, 0, 1) for name, holds in sizes(lib) if not holds]
    quant(lib, t=F64)
    text = lib.ep_last_error().decode()
    lib.ep_skip_rms_norm_grad_workspace_size(9, shp(3, 4), 2)
    kept = lib.ep_last_error().decode() == text and "quantize_mx8" in text
    print(json.dumps({"cases": len(got), "failures": bad + ([] if kept else [("a size query changed the last error", 0, 1)]),
                      "launches": int(lib.ep_kernel_launch_count())}))


if __name__ == "__main__":
    main()
