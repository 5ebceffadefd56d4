"""Host-side contract checks of GroupNorm and BiasDropout, run in a subprocess
with no visible CUDA device (CUDA_VISIBLE_DEVICES=""), as abi_host_cases.py: the
addresses are placeholders that nothing reads, and a case that passes the checks
ends in the device query (EP_ERR_CUDA)."""
import ctypes
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

F32, F16, BF16, F64 = 0, 1, 2, 7
OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4
A, B, C, D, E, F, G, H, I, J = (0x7F0000000000 + i * (1 << 36) for i in range(10))
BIG = 1 << 34   # workspace bytes


def shp(*d):
    return (ctypes.c_int64 * max(1, len(d)))(*d)


def gn(lib, t=F16, x=A, shape=(2, 3, 8), gamma=B, beta=C, groups=2, eps=1e-5, act=0, y=D, mean=None, inv=None,
       ws=E, wsb=BIG):
    return lib.ep_group_norm(t, x, None if shape is None else shp(*shape), gamma, beta, groups, eps, act, y, mean,
                             inv, ws, wsb, None)


def gng(lib, t=F16, dy=A, x=B, shape=(2, 3, 8), gamma=C, beta=D, groups=2, act=0, mean=E, inv=F, dx=G, dg=H, db=I,
        ws=J, wsb=BIG):
    return lib.ep_group_norm_grad(t, dy, x, None if shape is None else shp(*shape), gamma, beta, groups, act, mean,
                                  inv, dx, dg, db, ws, wsb, None)


def drop(lib, t=F16, x=A, shape=(4, 8), bias=B, res=C, ratio=0.1, seed=1, offset=2, od=None, y=D):
    return lib.ep_bias_dropout(t, x, None if shape is None else shp(*shape), len(shape or ()), bias, res, ratio, seed,
                               offset, od, y, None)


def dropg(lib, t=F16, dy=A, shape=(4, 8), ratio=0.1, od=None, dx=B, db=C, ws=D, wsb=BIG):
    return lib.ep_bias_dropout_grad(t, dy, shp(*shape), len(shape), ratio, 1, 2, od, dx, db, ws, wsb, None)


def cases(lib):
    wide = (1, 1 << 17, 256)   # 67 MB a sample: in no form held on chip, so with a workspace
    nan = float("nan")
    return [
        ("gn ok", gn(lib), CUDA), ("gn f32 ok", gn(lib, t=F32), CUDA), ("gn bf16 ok", gn(lib, t=BF16), CUDA),
        ("gn f64", gn(lib, t=F64), UNSUPPORTED),
        ("gn NULL shape", gn(lib, shape=None), INVALID),
        ("gn negative dim", gn(lib, shape=(2, -3, 8)), INVALID),
        ("gn overflowing dims", gn(lib, shape=(1 << 40, 1 << 20, 1 << 20)), INVALID),
        ("gn groups 0", gn(lib, groups=0), INVALID), ("gn groups -2", gn(lib, groups=-2), INVALID),
        ("gn groups do not divide", gn(lib, groups=3), INVALID),
        ("gn too many channels", gn(lib, shape=(1, 1, 1 << 25)), UNSUPPORTED),
        ("gn negative epsilon", gn(lib, eps=-1.0), INVALID), ("gn NaN epsilon", gn(lib, eps=nan), INVALID),
        ("gn epsilon 0 ok", gn(lib, eps=0.0), CUDA),
        ("gn SiLU ok", gn(lib, act=1), CUDA), ("gn activation 2", gn(lib, act=2), INVALID),
        ("gn activation -1", gn(lib, act=-1), INVALID),
        ("gn NULL X", gn(lib, x=None), INVALID), ("gn NULL gamma", gn(lib, gamma=None), INVALID),
        ("gn NULL Y", gn(lib, y=None), INVALID), ("gn NULL beta ok", gn(lib, beta=None), CUDA),
        ("gn misaligned X", gn(lib, x=A + 1), INVALID), ("gn misaligned f32 gamma", gn(lib, t=F32, gamma=B + 2), INVALID),
        ("gn f16 2-byte offset ok", gn(lib, x=A + 2), CUDA),
        ("gn misaligned mean", gn(lib, mean=F + 2), INVALID), ("gn misaligned inv", gn(lib, inv=F + 2), INVALID),
        ("gn statistics ok", gn(lib, mean=F, inv=G), CUDA),
        ("gn statistics overlap", gn(lib, mean=F, inv=F + 8), INVALID),
        ("gn mean overlaps X", gn(lib, mean=A), INVALID), ("gn inv overlaps Y", gn(lib, inv=D + 4), INVALID),
        ("gn in place ok", gn(lib, y=A), CUDA), ("gn partial overlap", gn(lib, y=A + 16), INVALID),
        ("gn Y overlaps gamma", gn(lib, y=B), INVALID), ("gn Y overlaps beta", gn(lib, y=C + 2), INVALID),
        ("gn empty N", gn(lib, shape=(0, 3, 8), x=None, gamma=None, y=None), OK),
        ("gn empty S", gn(lib, shape=(2, 0, 8), x=None, gamma=None, y=None), OK),
        ("gn empty still checks groups", gn(lib, shape=(0, 3, 8), groups=3), INVALID),
        ("gn no workspace", gn(lib, shape=wide, ws=None), WORKSPACE),
        ("gn small workspace", gn(lib, shape=wide, wsb=8), WORKSPACE),
        ("gn misaligned workspace", gn(lib, shape=wide, ws=E + 8), WORKSPACE),
        ("gn workspace overlaps X", gn(lib, shape=wide, ws=A), WORKSPACE),
        # --- gradient
        ("gng ok", gng(lib), CUDA), ("gng f64", gng(lib, t=F64), UNSUPPORTED),
        ("gng NULL shape", gng(lib, shape=None), INVALID), ("gng groups", gng(lib, groups=5), INVALID),
        ("gng activation", gng(lib, act=7), INVALID),
        ("gng NULL dY", gng(lib, dy=None), INVALID), ("gng NULL X", gng(lib, x=None), INVALID),
        ("gng NULL gamma", gng(lib, gamma=None), INVALID), ("gng NULL mean", gng(lib, mean=None), INVALID),
        ("gng NULL inv", gng(lib, inv=None), INVALID), ("gng NULL dX", gng(lib, dx=None), INVALID),
        ("gng NULL beta ok", gng(lib, beta=None), CUDA), ("gng no dgamma ok", gng(lib, dg=None), CUDA),
        ("gng no parameter gradients ok", gng(lib, dg=None, db=None), CUDA),
        ("gng misaligned dY", gng(lib, dy=A + 1), INVALID), ("gng misaligned mean", gng(lib, mean=E + 2), INVALID),
        ("gng misaligned dgamma", gng(lib, t=F32, dg=H + 2), INVALID),
        ("gng dX is dY ok", gng(lib, dx=A), CUDA), ("gng dX is X ok", gng(lib, dx=B), CUDA),
        ("gng dX overlaps dY", gng(lib, dx=A + 2), INVALID), ("gng dX overlaps gamma", gng(lib, dx=C), INVALID),
        ("gng dX overlaps mean", gng(lib, dx=E), INVALID),
        ("gng dgamma is gamma", gng(lib, dg=C), INVALID), ("gng dbeta is dgamma", gng(lib, db=H), INVALID),
        ("gng dbeta overlaps dX", gng(lib, db=G + 2), INVALID),
        ("gng no workspace", gng(lib, shape=wide, ws=None), WORKSPACE),
        ("gng small workspace", gng(lib, shape=wide, wsb=64), WORKSPACE),
        ("gng misaligned workspace", gng(lib, shape=wide, ws=J + 4), WORKSPACE),
        ("gng workspace overlaps dX", gng(lib, shape=wide, ws=G), WORKSPACE),
        ("gng empty without parameter gradients",
         gng(lib, shape=(0, 3, 8), dy=None, x=None, gamma=None, mean=None, inv=None, dx=None, dg=None, db=None), OK),
        # --- BiasDropout
        ("drop ok", drop(lib), CUDA), ("drop bf16 ok", drop(lib, t=BF16), CUDA), ("drop f64", drop(lib, t=F64), UNSUPPORTED),
        ("drop rank 0", drop(lib, shape=()), INVALID), ("drop rank 17", drop(lib, shape=(1,) * 17), UNSUPPORTED),
        ("drop NULL shape", lib.ep_bias_dropout(F16, A, None, 2, None, None, 0.1, 1, 2, None, D, None), INVALID),
        ("drop negative dim", drop(lib, shape=(4, -8)), INVALID),
        ("drop ratio 1", drop(lib, ratio=1.0), INVALID), ("drop ratio -0.1", drop(lib, ratio=-0.1), INVALID),
        ("drop ratio NaN", drop(lib, ratio=nan), INVALID), ("drop ratio 0 ok", drop(lib, ratio=0.0), CUDA),
        ("drop NULL X", drop(lib, x=None), INVALID), ("drop NULL Y", drop(lib, y=None), INVALID),
        ("drop no bias, no residual ok", drop(lib, bias=None, res=None), CUDA),
        ("drop misaligned bias", drop(lib, bias=B + 1), INVALID),
        ("drop misaligned offset_device", drop(lib, od=E + 4), INVALID), ("drop offset_device ok", drop(lib, od=E), CUDA),
        ("drop in place ok", drop(lib, y=A), CUDA), ("drop onto the residual ok", drop(lib, y=C), CUDA),
        ("drop Y overlaps X", drop(lib, y=A + 2), INVALID), ("drop Y overlaps bias", drop(lib, y=B), INVALID),
        ("drop Y overlaps offset_device", drop(lib, od=D + 8), INVALID),
        ("drop empty", drop(lib, shape=(0, 8), x=None, y=None, bias=None, res=None), OK),
        ("dropg ok", dropg(lib), CUDA), ("dropg f64", dropg(lib, t=F64), UNSUPPORTED),
        ("dropg ratio", dropg(lib, ratio=1.5), INVALID), ("dropg NULL dY", dropg(lib, dy=None), INVALID),
        ("dropg NULL dX", dropg(lib, dx=None), INVALID), ("dropg in place ok", dropg(lib, dx=A), CUDA),
        ("dropg dX overlaps dY", dropg(lib, dx=A + 2), INVALID), ("dropg dbias overlaps dX", dropg(lib, db=B), INVALID),
        ("dropg misaligned dbias", dropg(lib, db=C + 1), INVALID),
        ("dropg misaligned offset_device", dropg(lib, od=E + 4), INVALID),
        ("dropg no dbias, no workspace ok", dropg(lib, db=None, ws=None), CUDA),
        ("dropg no workspace", dropg(lib, ws=None), WORKSPACE), ("dropg small workspace", dropg(lib, wsb=8), WORKSPACE),
        ("dropg misaligned workspace", dropg(lib, ws=D + 8), WORKSPACE),
        ("dropg workspace overlaps dY", dropg(lib, ws=A), WORKSPACE),
        ("dropg empty without dbias", dropg(lib, shape=(0, 8), dy=None, dx=None, db=None), OK),
    ]


def main():
    assert os.environ.get("CUDA_VISIBLE_DEVICES", None) == "", "run with CUDA_VISIBLE_DEVICES=''"
    from transformer_epilogue_gb300 import _binding
    lib = _binding.load_library()
    n0 = lib.ep_kernel_launch_count()
    bad, ran = [], cases(lib)
    for name, got, want in ran:
        if got != want:
            bad.append((name, got, want))
    # size queries: host arithmetic; 0 for what the calls reject, and errors stay as they were
    before = lib.ep_last_error()
    for name, got in (("gn", lib.ep_group_norm_workspace_size(F16, shp(2, 3, 8), 3)),
                      ("gng", lib.ep_group_norm_grad_workspace_size(F64, shp(2, 3, 8), 2)),
                      ("drop", lib.ep_bias_dropout_grad_workspace_size(F16, shp(4, -8), 2)),
                      ("gn empty", lib.ep_group_norm_workspace_size(F16, shp(0, 3, 8), 2))):
        if got != 0:
            bad.append(("workspace size " + name, got, 0))
    if lib.ep_last_error() != before:
        bad.append(("last error moved", 1, 0))
    # a training batch's workspace stays a small share of its data
    for shape, groups in (((16, 1024, 4096), 32), ((8192, 1, 2048), 16), ((1, 1 << 20, 128), 32), ((2, 4096, 640), 32)):
        n = shape[0] * shape[1] * shape[2] * 2
        w = max(lib.ep_group_norm_workspace_size(F16, shp(*shape), groups),
                lib.ep_group_norm_grad_workspace_size(F16, shp(*shape), groups),
                lib.ep_bias_dropout_grad_workspace_size(F16, shp(*shape), 3))
        if w > max(n // 2, 1 << 22):
            bad.append(("workspace of %r" % (shape,), w, n // 2))
    if lib.ep_kernel_launch_count() != n0:
        bad.append(("launch count moved", lib.ep_kernel_launch_count(), n0))
    print(json.dumps({"cases": len(ran), "failures": bad}))
    return 1 if bad else 0


if __name__ == "__main__":
    sys.exit(main())
