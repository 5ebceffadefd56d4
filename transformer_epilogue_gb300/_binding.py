"""Thin ctypes binding of the C ABI declared in ``include/ep.h``.

Argument marshalling only: every function here checks that its tensors are
contiguous CUDA tensors, allocates outputs the caller did not pass (PyTorch is
the allocator), and calls the C entry point of the same name on the current
CUDA stream.  All computation happens in the library's CUDA kernels; there is
no CPU or PyTorch fallback.  A non-OK status raises ``EpError``.  Nothing here is
recorded for autograd: outputs are detached whatever the inputs require, and the
``_grad`` functions are called by hand (or from a ``torch.autograd.Function``).
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "lib", "libtransformer_epilogue.so")

EP_F32, EP_F16, EP_BF16 = 0, 1, 2
EP_OK, EP_ERR_INVALID_ARG, EP_ERR_UNSUPPORTED, EP_ERR_WORKSPACE, EP_ERR_CUDA = 0, 1, 2, 3, 4
STATUS_NAMES = {0: "EP_OK", 1: "EP_ERR_INVALID_ARG", 2: "EP_ERR_UNSUPPORTED", 3: "EP_ERR_WORKSPACE",
                4: "EP_ERR_CUDA"}

EP_ACT_NONE, EP_ACT_SILU, EP_ACT_RELU, EP_ACT_QUICK_GELU, EP_ACT_GELU, EP_ACT_FAST_GELU = 0, 1, 2, 3, 4, 5

# Attribute defaults of the op definitions (manifest `attributes` sections).
DEFAULT_EPSILON = 9.999999960041972e-13   # SkipLayerNormalization
DEFAULT_ALPHA = 1.702                     # QuickGelu
DEFAULT_AXIS = 1                          # BiasSoftmax
DEFAULT_GROUP_NORM_EPSILON = 1e-5         # GroupNorm (contrib op schema)

_TORCH_TO_EP = {torch.float32: EP_F32, torch.float16: EP_F16, torch.bfloat16: EP_BF16}

_lib = None

_i64p = ctypes.POINTER(ctypes.c_int64)
_vp = ctypes.c_void_p
_i64 = ctypes.c_int64

# name -> (restype, argtypes)
_SIGNATURES = {
    "ep_last_error": (ctypes.c_char_p, []),
    "ep_status_name": (ctypes.c_char_p, [ctypes.c_int]),
    "ep_kernel_launch_count": (ctypes.c_uint64, []),
    "ep_abi_version": (ctypes.c_int, []),
    "ep_pipeline_timeouts": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint64), ctypes.c_int]),
    "ep_selftest_bounded_wait": (ctypes.c_int, [ctypes.c_uint32, ctypes.POINTER(ctypes.c_uint64), _vp]),
    "ep_skip_layer_norm": (ctypes.c_int, [ctypes.c_int, _vp, _i64p, ctypes.c_int, _vp, _i64p, ctypes.c_int,
                                          _vp, _vp, _vp, ctypes.c_float, _vp, _vp, _vp]),
    "ep_skip_layer_norm_ex": (ctypes.c_int, [ctypes.c_int, _vp, _i64p, ctypes.c_int, _vp, _i64p, ctypes.c_int,
                                             _vp, _vp, _vp, ctypes.c_float, ctypes.c_int, _vp, _vp, _vp, _vp,
                                             _vp]),
    "ep_bias_softmax": (ctypes.c_int, [ctypes.c_int, _vp, _i64p, ctypes.c_int, _vp, ctypes.c_int64,
                                       ctypes.c_int, ctypes.c_int, _vp, _vp, ctypes.c_size_t, _vp]),
    "ep_bias_softmax_workspace_size": (ctypes.c_size_t, [ctypes.c_int, _i64p, ctypes.c_int, ctypes.c_int]),
    "ep_bias_softmax_noalloc": (ctypes.c_int, [ctypes.c_int, _vp, _i64p, ctypes.c_int, _vp, ctypes.c_int64,
                                               ctypes.c_int, ctypes.c_int, _vp, _vp]),
    "ep_bias_add": (ctypes.c_int, [ctypes.c_int, _vp, _i64p, _vp, _vp, _vp, _vp]),
    "ep_quick_gelu": (ctypes.c_int, [ctypes.c_int, _vp, ctypes.c_int64, ctypes.c_float, _vp, _vp]),
    "ep_group_norm": (ctypes.c_int, [ctypes.c_int, _vp, _i64p, _vp, _vp, ctypes.c_int64, ctypes.c_float,
                                     ctypes.c_int, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "ep_group_norm_workspace_size": (ctypes.c_size_t, [ctypes.c_int, _i64p, ctypes.c_int64]),
    "ep_group_norm_workspace_size_aligned": (ctypes.c_size_t, [ctypes.c_int, _i64p, ctypes.c_int64]),
    "ep_group_norm_grad": (ctypes.c_int, [ctypes.c_int, _vp, _vp, _i64p, _vp, _vp, ctypes.c_int64, ctypes.c_int,
                                          _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "ep_group_norm_grad_workspace_size": (ctypes.c_size_t, [ctypes.c_int, _i64p, ctypes.c_int64]),
    "ep_group_norm_grad_workspace_size_aligned": (ctypes.c_size_t, [ctypes.c_int, _i64p, ctypes.c_int64]),
    "ep_bias_dropout": (ctypes.c_int, [ctypes.c_int, _vp, _i64p, ctypes.c_int, _vp, _vp, ctypes.c_double,
                                       ctypes.c_uint64, ctypes.c_uint64, _vp, _vp, _vp]),
    "ep_bias_dropout_grad": (ctypes.c_int, [ctypes.c_int, _vp, _i64p, ctypes.c_int, ctypes.c_double,
                                            ctypes.c_uint64, ctypes.c_uint64, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                            _vp]),
    "ep_bias_dropout_grad_workspace_size": (ctypes.c_size_t, [ctypes.c_int, _i64p, ctypes.c_int]),
    "ep_quantize_mx8": (ctypes.c_int, [ctypes.c_int, _vp, _i64p, ctypes.c_int, _vp, _vp, _vp]),
    "ep_dequantize_mx8": (ctypes.c_int, [ctypes.c_int, _vp, _vp, _i64p, ctypes.c_int, _vp, _vp]),
    "ep_skip_rms_norm_mx8": (ctypes.c_int, [ctypes.c_int, _vp, _i64p, ctypes.c_int, _vp, _vp, _vp, ctypes.c_float,
                                            _vp, _vp, _vp, _vp, _vp]),
    "ep_skip_rms_norm_grad": (ctypes.c_int, [ctypes.c_int, _vp, _vp, _i64p, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp,
                                             _vp, ctypes.c_size_t, _vp]),
    "ep_skip_rms_norm_grad_workspace_size": (ctypes.c_size_t, [ctypes.c_int, _i64p, ctypes.c_int]),
    "ep_matmul_bias_act": (ctypes.c_int, [ctypes.c_int, _vp, _vp, _i64, _i64, _i64, _vp, _vp, ctypes.c_int,
                                          ctypes.c_float, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "ep_matmul_bias_act_mx8": (ctypes.c_int, [ctypes.c_int, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp,
                                              ctypes.c_int, ctypes.c_float, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "ep_matmul_bias_act_workspace_size": (ctypes.c_size_t, [ctypes.c_int, _i64, _i64, _i64, ctypes.c_int]),
    "ep_matmul_bias_act_grad": (ctypes.c_int, [ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                               ctypes.c_int, ctypes.c_float, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "ep_matmul_bias_act_grad_workspace_size": (ctypes.c_size_t, [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int,
                                                                 ctypes.c_int]),
}


class EpError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def load_library(path: str = LIB_PATH):
    """Load the C-ABI library (built by ``__graft_entry__.build()`` or
    ``python -m transformer_epilogue_gb300.build``).  Raises if it is missing:
    there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"CUDA library not built: {path} is missing "
                          "(run `python -m transformer_epilogue_gb300.build`)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def raw():
    """The loaded ctypes library (for pointer-level calls)."""
    return load_library()


def _check(status: int):
    if status != EP_OK:
        msg = load_library().ep_last_error().decode(errors="replace")
        raise EpError(status, msg)


def _shape(dims) -> ctypes.Array:
    dims = [int(d) for d in dims]
    return (ctypes.c_int64 * max(1, len(dims)))(*dims)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype(t: torch.Tensor) -> int:
    try:
        return _TORCH_TO_EP[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _cuda(name, t, optional=False):
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def kernel_launch_count() -> int:
    return int(load_library().ep_kernel_launch_count())


def ep_pipeline_timeouts(clear=False) -> int:
    """Bounded-wait timeouts the staged kernels counted on the current device
    (synchronises with the device)."""
    n = ctypes.c_uint64(0)
    _check(load_library().ep_pipeline_timeouts(ctypes.byref(n), int(bool(clear))))
    return int(n.value)


def ep_selftest_bounded_wait(timeout_us=5000, stream=None) -> int:
    """Run the failure-detection self-test; returns the timed-out waits counted
    meanwhile (1 when the mechanism works)."""
    n = ctypes.c_uint64(0)
    _check(load_library().ep_selftest_bounded_wait(int(timeout_us), ctypes.byref(n),
                                                   _stream(stream, torch.cuda.current_device())))
    return int(n.value)


def ep_skip_layer_norm(input, skip, gamma, beta=None, bias=None, epsilon=DEFAULT_EPSILON, output=None,
                       input_skip_bias_sum=None, stream=None):
    """SkipLayerNormalization.  ``input_skip_bias_sum``: a tensor to fill, True
    to allocate one, or None.  Returns (output, input_skip_bias_sum or None)."""
    lib = load_library()
    for n, t in (("input", input), ("skip", skip), ("gamma", gamma)):
        _cuda(n, t)
    _cuda("beta", beta, True)
    _cuda("bias", bias, True)
    if output is None:
        output = torch.empty_like(input)
    _cuda("output", output)
    if input_skip_bias_sum is True:
        input_skip_bias_sum = torch.empty_like(input)
    elif input_skip_bias_sum is False:
        input_skip_bias_sum = None
    _cuda("input_skip_bias_sum", input_skip_bias_sum, True)
    st = lib.ep_skip_layer_norm(_dtype(input), _ptr(input), _shape(input.shape), input.dim(),
                                _ptr(skip), _shape(skip.shape), skip.dim(),
                                _ptr(gamma), _ptr(beta), _ptr(bias), float(epsilon),
                                _ptr(output), _ptr(input_skip_bias_sum), _stream(stream, input.device))
    _check(st)
    return output, input_skip_bias_sum


def ep_skip_layer_norm_ex(input, skip, gamma, beta=None, bias=None, epsilon=DEFAULT_EPSILON, simplified=False,
                          output=None, input_skip_bias_sum=None, mean=None, inv_std_dev=None, stream=None):
    """SkipLayerNormalization with the RMS form (``simplified``) and the
    per-row float32 statistics.  ``mean`` / ``inv_std_dev``: tensors to fill,
    True to allocate, or None.  Returns (output, input_skip_bias_sum, mean,
    inv_std_dev), the last three None when not requested."""
    lib = load_library()
    for n, t in (("input", input), ("skip", skip), ("gamma", gamma)):
        _cuda(n, t)
    _cuda("beta", beta, True)
    _cuda("bias", bias, True)
    if output is None:
        output = torch.empty_like(input)
    _cuda("output", output)
    if input_skip_bias_sum is True:
        input_skip_bias_sum = torch.empty_like(input)
    elif input_skip_bias_sum is False:
        input_skip_bias_sum = None
    _cuda("input_skip_bias_sum", input_skip_bias_sum, True)
    rows = input.numel() // max(1, input.shape[-1])
    stat_shape = tuple(input.shape[:-1]) + (1,)
    if mean is True:
        mean = torch.empty(stat_shape, dtype=torch.float32, device=input.device)
    if inv_std_dev is True:
        inv_std_dev = torch.empty(stat_shape, dtype=torch.float32, device=input.device)
    for n, t in (("mean", mean), ("inv_std_dev", inv_std_dev)):
        _cuda(n, t, True)
        if t is not None and (t.dtype != torch.float32 or t.numel() != rows):
            raise ValueError(f"{n} must be a float32 tensor of {rows} elements")
    st = lib.ep_skip_layer_norm_ex(_dtype(input), _ptr(input), _shape(input.shape), input.dim(),
                                   _ptr(skip), _shape(skip.shape), skip.dim(),
                                   _ptr(gamma), _ptr(beta), _ptr(bias), float(epsilon), int(bool(simplified)),
                                   _ptr(output), _ptr(input_skip_bias_sum), _ptr(mean), _ptr(inv_std_dev),
                                   _stream(stream, input.device))
    _check(st)
    return output, input_skip_bias_sum, mean, inv_std_dev


def ep_bias_softmax_workspace_size(dtype, shape, axis=DEFAULT_AXIS) -> int:
    lib = load_library()
    code = _TORCH_TO_EP[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(lib.ep_bias_softmax_workspace_size(code, _shape(shape), len(shape), int(axis)))


def ep_bias_softmax(data, bias, axis=DEFAULT_AXIS, is_inner_broadcast=None, output=None, workspace=None,
                    stream=None):
    """BiasSoftmax.  ``is_inner_broadcast`` is required (the op definition has
    no default for it).  A workspace is allocated when the split-row path needs
    one and none is passed.  Returns output."""
    if is_inner_broadcast is None:
        raise ValueError("is_inner_broadcast is required")
    lib = load_library()
    _cuda("data", data)
    _cuda("bias", bias)
    if output is None:
        output = torch.empty_like(data)
    _cuda("output", output)
    need = ep_bias_softmax_workspace_size(data.dtype, data.shape, axis) if data.dtype in _TORCH_TO_EP else 0
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=data.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.ep_bias_softmax(_dtype(data), _ptr(data), _shape(data.shape), data.dim(), _ptr(bias),
                             int(bias.numel()), int(axis), int(is_inner_broadcast), _ptr(output),
                             _ptr(workspace), wbytes, _stream(stream, data.device))
    _check(st)
    return output


def ep_bias_softmax_noalloc(data, bias, axis=DEFAULT_AXIS, is_inner_broadcast=None, output=None, stream=None):
    """BiasSoftmax for callers that cannot allocate device memory: the
    split-row scratch comes from a fixed 1 MiB array inside the library
    (rows * ceil(blockSize / chunk) <= 131072 when blockSize > 16384, chunk =
    4096 for float32, 8192 for float16/bfloat16).  Calls
    that may overlap on the GPU share that array and must be ordered by the
    caller.  Pass ``output`` to keep the call free of allocations (otherwise
    PyTorch allocates it here).  Returns output."""
    if is_inner_broadcast is None:
        raise ValueError("is_inner_broadcast is required")
    lib = load_library()
    _cuda("data", data)
    _cuda("bias", bias)
    if output is None:
        output = torch.empty_like(data)
    _cuda("output", output)
    st = lib.ep_bias_softmax_noalloc(_dtype(data), _ptr(data), _shape(data.shape), data.dim(), _ptr(bias),
                                     int(bias.numel()), int(axis), int(is_inner_broadcast), _ptr(output),
                                     _stream(stream, data.device))
    _check(st)
    return output


def ep_bias_add(X, bias, skip, Y=None, stream=None):
    """BiasAdd on (N, S, C) tensors.  Returns Y."""
    lib = load_library()
    for n, t in (("X", X), ("bias", bias), ("skip", skip)):
        _cuda(n, t)
    if X.dim() != 3:
        raise ValueError("X must have rank 3 (N, S, C)")
    if tuple(skip.shape) != tuple(X.shape) or bias.numel() != X.shape[2] or bias.dim() != 1:
        raise ValueError("skip must match X and bias must have C elements")
    if Y is None:
        Y = torch.empty_like(X)
    _cuda("Y", Y)
    if tuple(Y.shape) != tuple(X.shape):
        raise ValueError("Y must match X")
    st = lib.ep_bias_add(_dtype(X), _ptr(X), _shape(X.shape), _ptr(bias), _ptr(skip), _ptr(Y),
                         _stream(stream, X.device))
    _check(st)
    return Y


def ep_quick_gelu(X, alpha=DEFAULT_ALPHA, Y=None, stream=None):
    """QuickGelu over all elements of X.  Returns Y."""
    lib = load_library()
    _cuda("X", X)
    if Y is None:
        Y = torch.empty_like(X)
    _cuda("Y", Y)
    if Y.numel() != X.numel():
        raise ValueError("Y must have as many elements as X")
    st = lib.ep_quick_gelu(_dtype(X), _ptr(X), int(X.numel()), float(alpha), _ptr(Y), _stream(stream, X.device))
    _check(st)
    return Y


# ---------------------------------------------------------------------------
# GroupNorm and BiasDropout, with their gradients.  Operands are checked against
# the first one (device, dtype, shape) before their addresses are passed on.  The
# calls run on the current stream, or with `stream` current, so that what is
# allocated here (outputs, a workspace) belongs to the stream it is used on.
# Small calls cost what the host costs: shape arrays and workspace sizes are
# kept by value (shape, dtype), and the checks take a few attribute reads.
# ---------------------------------------------------------------------------

# the current stream's handle without a Stream object (2 us less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _first(name, t):
    """The operand that the others are checked against: its device index and dtype code."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.get_device(), _dtype(t)


def _operand(name, t, like, index, shape=None, dtype=None):
    """t, checked to be a contiguous CUDA tensor on like's device (`index`) with
    the given dtype (like's if None) and shape (any if None)."""
    dtype = like.dtype if dtype is None else dtype
    if isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype and \
            (shape is None or t.shape == shape) and t.is_contiguous():
        return t
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must have dtype {dtype}, not {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _elsewhere(stream, index):
    """None if the call can run as it is, on the current stream of the current
    device; else a context in which it can."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"the stream belongs to {stream.device}, the tensors to cuda:{index}")
        return torch.cuda.stream(stream)
    return None if _current_device() == index else torch.cuda.device(index)


# Scratch comes from PyTorch's allocator as a bare pointer: a tensor that nobody
# sees costs 2 us more.
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc",
                     lambda size, stream: torch.cuda.caching_allocator_alloc(size, stream=stream))
_raw_delete = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", torch.cuda.caching_allocator_delete)


def _scratch(workspace, need, like, raw_stream):
    """(pointer, bytes, owned): the caller's workspace, or memory allocated for
    this call, which goes back to the allocator once the call is in the stream
    (owned; the current device and stream are the call's)."""
    if workspace is None:
        if need == 0:
            return None, 0, False
        return _raw_alloc(need, raw_stream), need, True
    if not workspace.is_cuda or workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on the operands' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), False


def _addr(t):
    return None if t is None else t.data_ptr()


def _u64(name, v):
    v = int(v)
    if not 0 <= v < 1 << 64:
        raise ValueError(f"{name} must be an unsigned 64-bit number")
    return v


@functools.lru_cache(maxsize=4096)
def _dims(shape):
    """A shape as the C array that the library reads."""
    return _shape(shape)


def _nsc(shape):
    """(N, S, C) of a channels-last shape: the dimensions between the first and
    the last are positions."""
    if len(shape) < 3:
        raise ValueError("X must have the shape (N, positions..., C)")
    s = 1
    for d in shape[1:-1]:
        s *= d
    return _shape((shape[0], s, shape[-1]))


@functools.lru_cache(maxsize=4096)
def _group_norm_plan(code, shape, groups, grad):
    """(N, S, C) as the library reads it, the channels' shape, and the workspace's
    bytes for tensors anywhere and on 16-byte boundaries."""
    lib = load_library()
    name = "ep_group_norm_grad_workspace_size" if grad else "ep_group_norm_workspace_size"
    nsc = _nsc(shape)
    return (nsc, torch.Size(shape[-1:]), int(getattr(lib, name)(code, nsc, groups)),
            int(getattr(lib, name + "_aligned")(code, nsc, groups)))


@functools.lru_cache(maxsize=4096)
def _bias_dropout_grad_need(code, shape):
    return int(load_library().ep_bias_dropout_grad_workspace_size(code, _dims(shape), len(shape)))


def _code(dtype):
    return _TORCH_TO_EP[dtype] if isinstance(dtype, torch.dtype) else int(dtype)


def ep_group_norm_workspace_size(dtype, shape, groups, aligned=False) -> int:
    """Workspace bytes of ep_group_norm for a channels-last shape.  ``aligned``: X
    and Y start on 16-byte boundaries (0 for small samples and tokens)."""
    return _group_norm_plan(_code(dtype), tuple(shape), int(groups), False)[3 if aligned else 2]


def ep_group_norm_grad_workspace_size(dtype, shape, groups, aligned=False) -> int:
    """Workspace bytes of ep_group_norm_grad for a channels-last shape.  ``aligned``:
    dY, X and dX start on 16-byte boundaries."""
    return _group_norm_plan(_code(dtype), tuple(shape), int(groups), True)[3 if aligned else 2]


def ep_bias_dropout_grad_workspace_size(dtype, shape) -> int:
    """Workspace bytes of ep_bias_dropout_grad with dbias."""
    return _bias_dropout_grad_need(_code(dtype), tuple(shape))


def _group_stats(name, t, X, index, n, groups):
    if t is None or t is False:
        return None
    if t is True:
        return torch.empty((n, max(0, groups)), dtype=torch.float32, device=X.device)
    _operand(name, t, X, index, dtype=torch.float32)
    if t.numel() != n * groups:
        raise ValueError(f"{name} must have {n * groups} elements")
    return t


def _param_grad(name, t, X, index, channels):
    if t is None or t is False:
        return None
    if t is True:
        return torch.empty(channels, dtype=X.dtype, device=X.device)
    return _operand(name, t, X, index, channels)


def ep_group_norm(X, gamma, beta=None, groups=None, epsilon=DEFAULT_GROUP_NORM_EPSILON, activation=EP_ACT_NONE,
                  Y=None, mean=None, inv_std_dev=None, workspace=None, stream=None):
    """GroupNorm of a channels-last X (N, positions..., C), optionally followed
    by a SiLU (``EP_ACT_SILU``).  Tokens (N, C) are passed as ``X[:, None]``.  Not
    recorded for autograd: see ``ep_group_norm_grad``.  ``groups`` is required (the op definition has
    no default for it).  ``mean`` / ``inv_std_dev``: float32 tensors of
    N * groups elements to fill, True to allocate (N, groups), or None.
    Returns (Y, mean, inv_std_dev), the last two None when not requested."""
    if groups is None:
        raise ValueError("groups is required")
    index, code = _first("X", X)
    other = _elsewhere(stream, index)
    if other is not None:
        with other:
            return ep_group_norm(X, gamma, beta, groups, epsilon, activation, Y, mean, inv_std_dev, workspace)
    lib = load_library()
    shape, groups = X.shape, int(groups)
    nsc, channels, need, need_aligned = _group_norm_plan(code, shape, groups, False)
    _operand("gamma", gamma, X, index, channels)
    if beta is not None:
        _operand("beta", beta, X, index, channels)
    Y = torch.empty_like(X) if Y is None else _operand("Y", Y, X, index, shape)
    mean = _group_stats("mean", mean, X, index, shape[0], groups)
    inv_std_dev = _group_stats("inv_std_dev", inv_std_dev, X, index, shape[0], groups)
    px, py = X.data_ptr(), Y.data_ptr()
    if (px | py) & 15 == 0:
        need = need_aligned
    args = (code, px, nsc, gamma.data_ptr(), _addr(beta), groups, float(epsilon), int(activation), py, _addr(mean),
            _addr(inv_std_dev))
    s = _raw_stream(index)
    ws, wbytes, owned = _scratch(workspace, need, X, s)
    try:
        _check(lib.ep_group_norm(*args, ws, wbytes, s))
    finally:
        if owned:
            _raw_delete(ws)
    return Y, mean, inv_std_dev


def ep_group_norm_grad(dY, X, gamma, beta, mean, inv_std_dev, groups=None, activation=EP_ACT_NONE, dX=None,
                       dgamma=True, dbeta=True, workspace=None, stream=None):
    """Gradient of ep_group_norm, from the statistics it returned (``beta``: None
    where the forward call had none).  ``dgamma`` / ``dbeta``: tensors to fill,
    True to allocate, or None.  Returns (dX, dgamma, dbeta), the last two None
    when not requested."""
    if groups is None:
        raise ValueError("groups is required")
    index, code = _first("X", X)
    other = _elsewhere(stream, index)
    if other is not None:
        with other:
            return ep_group_norm_grad(dY, X, gamma, beta, mean, inv_std_dev, groups, activation, dX, dgamma, dbeta,
                                      workspace)
    lib = load_library()
    shape, groups = X.shape, int(groups)
    nsc, channels, need, need_aligned = _group_norm_plan(code, shape, groups, True)
    _operand("dY", dY, X, index, shape)
    _operand("gamma", gamma, X, index, channels)
    if beta is not None:
        _operand("beta", beta, X, index, channels)
    for name, t in (("mean", mean), ("inv_std_dev", inv_std_dev)):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} is required")
        _group_stats(name, t, X, index, shape[0], groups)
    dX = torch.empty_like(X) if dX is None else _operand("dX", dX, X, index, shape)
    dgamma = _param_grad("dgamma", dgamma, X, index, channels)
    dbeta = _param_grad("dbeta", dbeta, X, index, channels)
    pdy, px, pdx = dY.data_ptr(), X.data_ptr(), dX.data_ptr()
    if (pdy | px | pdx) & 15 == 0:
        need = need_aligned
    args = (code, pdy, px, nsc, gamma.data_ptr(), _addr(beta), groups, int(activation), mean.data_ptr(),
            inv_std_dev.data_ptr(), pdx, _addr(dgamma), _addr(dbeta))
    s = _raw_stream(index)
    ws, wbytes, owned = _scratch(workspace, need, X, s)
    try:
        _check(lib.ep_group_norm_grad(*args, ws, wbytes, s))
    finally:
        if owned:
            _raw_delete(ws)
    return dX, dgamma, dbeta


def _offset_device(t, like):
    """A device number added to the offset: one int64 or uint64 element."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != like.device or t.numel() != 1 \
            or t.dtype not in (torch.int64, torch.uint64):
        raise ValueError("offset_device must be one int64 or uint64 element on the operands' device")
    return t.data_ptr()


def ep_bias_dropout(X, ratio, seed, offset=0, bias=None, residual=None, offset_device=None, Y=None, stream=None):
    """BiasDropout: residual + keep * (X + bias) / (1 - ratio), the mask made
    from (seed, offset) and the element's index.  Not recorded for autograd: see
    ``ep_bias_dropout_grad``.  ``offset_device``: a one-element
    int64 CUDA tensor added to ``offset`` when the kernel runs (for captured
    graphs).  Returns Y."""
    index, code = _first("X", X)
    other = _elsewhere(stream, index)
    if other is not None:
        with other:
            return ep_bias_dropout(X, ratio, seed, offset, bias, residual, offset_device, Y)
    lib = load_library()
    shape = X.shape
    if bias is not None:
        _operand("bias", bias, X, index, shape[-1:])
    if residual is not None:
        _operand("residual", residual, X, index, shape)
    od = _offset_device(offset_device, X)
    Y = torch.empty_like(X) if Y is None else _operand("Y", Y, X, index, shape)
    _check(lib.ep_bias_dropout(code, X.data_ptr(), _dims(shape), len(shape), _addr(bias), _addr(residual), float(ratio),
                               _u64("seed", seed), _u64("offset", offset), od, Y.data_ptr(), _raw_stream(index)))
    return Y


def ep_bias_dropout_grad(dY, ratio, seed, offset=0, offset_device=None, dX=None, dbias=None, workspace=None,
                         stream=None):
    """Gradient of ep_bias_dropout (the residual's is dY itself).  ``dbias``: a
    tensor to fill, True to allocate, or None.  Returns (dX, dbias or None)."""
    index, code = _first("dY", dY)
    other = _elsewhere(stream, index)
    if other is not None:
        with other:
            return ep_bias_dropout_grad(dY, ratio, seed, offset, offset_device, dX, dbias, workspace)
    lib = load_library()
    shape = dY.shape
    od = _offset_device(offset_device, dY)
    dX = torch.empty_like(dY) if dX is None else _operand("dX", dX, dY, index, shape)
    dbias = _param_grad("dbias", dbias, dY, index, shape[-1:])
    need = 0 if dbias is None else _bias_dropout_grad_need(code, shape)
    args = (code, dY.data_ptr(), _dims(shape), len(shape), float(ratio), _u64("seed", seed), _u64("offset", offset),
            od, dX.data_ptr(), _addr(dbias))
    s = _raw_stream(index)
    ws, wbytes, owned = _scratch(workspace, need, dY, s)
    try:
        _check(lib.ep_bias_dropout_grad(*args, ws, wbytes, s))
    finally:
        if owned:
            _raw_delete(ws)
    return dX, dbias


# ---------------------------------------------------------------------------
# MX8 (rows in 8 bits: torch.float8_e4m3fn elements, a torch.float8_e8m0fnu scale
# for each 32 of a row), the RMS norm and the matrix product.  Checks, streams and
# allocations as above.
# ---------------------------------------------------------------------------

_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu

# What follows from a shape, a device index or the sizes of a product is kept by value.


@functools.lru_cache(maxsize=64)
def _cuda_device(index):
    return torch.device("cuda", index)


@functools.lru_cache(maxsize=4096)
def _rows_plan(shape):
    """Rows along the last dimension: the C array, the rank, the shapes of a parameter, of MX8 scales and of a
    statistic for each row."""
    if len(shape) == 0:
        raise ValueError("rows need a dimension")
    return (_shape(shape), len(shape), torch.Size(shape[-1:]), torch.Size(shape[:-1] + ((shape[-1] + 31) // 32,)),
            torch.Size(shape[:-1] + (1,)))


def _scale_shape(shape):
    return _rows_plan(shape)[3]


def _mx8_out(name, Q, scales, like, index, shape, scale_shape):
    """Elements and scales to fill, made where they are not given."""
    if Q is None and scales is None:
        device = _cuda_device(index)
        return (torch.empty(shape, dtype=_E4M3, device=device), torch.empty(scale_shape, dtype=_E8M0, device=device))
    if Q is None or scales is None:
        raise ValueError(f"{name} and its scales are given together")
    return (_operand(name, Q, like, index, shape, _E4M3),
            _operand(f"{name}'s scales", scales, like, index, scale_shape, _E8M0))


def ep_quantize_mx8(X, Q=None, scales=None, stream=None):
    """X's rows (along its last dimension) in MX8.  Returns (Q, scales):
    float8_e4m3fn of X's shape, and a float8_e8m0fnu scale for each 32 of a row."""
    index, code = _first("X", X)
    other = _elsewhere(stream, index)
    if other is not None:
        with other:
            return ep_quantize_mx8(X, Q, scales)
    shape = X.shape
    dims, rank, _, scale_shape, _ = _rows_plan(shape)
    Q, scales = _mx8_out("Q", Q, scales, X, index, shape, scale_shape)
    _check(load_library().ep_quantize_mx8(code, X.data_ptr(), dims, rank, Q.data_ptr(), scales.data_ptr(),
                                          _raw_stream(index)))
    return Q, scales


def _mx8_in(name, Q, scales):
    if not isinstance(Q, torch.Tensor) or not Q.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    index = Q.get_device()
    _operand(name, Q, Q, index, dtype=_E4M3)
    _operand(f"{name}'s scales", scales, Q, index, _scale_shape(Q.shape), _E8M0)
    return index


def ep_dequantize_mx8(Q, scales, dtype=None, Y=None, stream=None):
    """The values of MX8 rows as ``dtype`` (or Y's).  Returns Y."""
    index = _mx8_in("Q", Q, scales)
    if Y is None and dtype is None:
        raise ValueError("dtype or Y is required")
    other = _elsewhere(stream, index)
    if other is not None:
        with other:
            return ep_dequantize_mx8(Q, scales, dtype, Y)
    shape = Q.shape
    if Y is None:
        Y = torch.empty(shape, dtype=dtype, device=_cuda_device(index))
    else:
        _operand("Y", Y, Q, index, shape, Y.dtype if dtype is None else dtype)
    _check(load_library().ep_dequantize_mx8(_dtype(Y), Q.data_ptr(), scales.data_ptr(), _dims(shape), len(shape),
                                            Y.data_ptr(), _raw_stream(index)))
    return Y


def _row_stats(name, t, X, index, stat_shape):
    if t is True:
        return torch.empty(stat_shape, dtype=torch.float32, device=_cuda_device(index))
    if t is None or t is False:
        return None
    _operand(name, t, X, index, dtype=torch.float32)
    if t.numel() != stat_shape.numel():
        raise ValueError(f"{name} must have {stat_shape.numel()} elements")
    return t


def ep_skip_rms_norm_mx8(input, skip, gamma, bias=None, epsilon=DEFAULT_EPSILON, Q=None, scales=None,
                         input_skip_bias_sum=None, inv_std_dev=None, stream=None):
    """RMS norm of (input + skip) + bias to MX8 rows; ``skip`` has input's shape or
    is None.  ``input_skip_bias_sum`` / ``inv_std_dev``: a tensor to fill (the sum may
    be input or skip), True to allocate one, or None.  Returns (Q, scales,
    input_skip_bias_sum, inv_std_dev), the last two None when not requested."""
    index, code = _first("input", input)
    other = _elsewhere(stream, index)
    if other is not None:
        with other:
            return ep_skip_rms_norm_mx8(input, skip, gamma, bias, epsilon, Q, scales, input_skip_bias_sum, inv_std_dev)
    shape = input.shape
    dims, rank, channels, scale_shape, stat_shape = _rows_plan(shape)
    if skip is not None:
        _operand("skip", skip, input, index, shape)
    _operand("gamma", gamma, input, index, channels)
    if bias is not None:
        _operand("bias", bias, input, index, channels)
    Q, scales = _mx8_out("Q", Q, scales, input, index, shape, scale_shape)
    if input_skip_bias_sum is True:
        input_skip_bias_sum = torch.empty_like(input)
    elif input_skip_bias_sum is False:
        input_skip_bias_sum = None
    if input_skip_bias_sum is not None:
        _operand("input_skip_bias_sum", input_skip_bias_sum, input, index, shape)
    inv_std_dev = _row_stats("inv_std_dev", inv_std_dev, input, index, stat_shape)
    _check(load_library().ep_skip_rms_norm_mx8(
        code, input.data_ptr(), dims, rank, _addr(skip), gamma.data_ptr(), _addr(bias), float(epsilon),
        Q.data_ptr(), scales.data_ptr(), _addr(input_skip_bias_sum), _addr(inv_std_dev), _raw_stream(index)))
    return Q, scales, input_skip_bias_sum, inv_std_dev


@functools.lru_cache(maxsize=4096)
def _rms_norm_grad_need(code, shape):
    return int(load_library().ep_skip_rms_norm_grad_workspace_size(code, _dims(shape), len(shape)))


def ep_skip_rms_norm_grad_workspace_size(dtype, shape) -> int:
    """Workspace bytes of ep_skip_rms_norm_grad."""
    return _rms_norm_grad_need(_code(dtype), tuple(shape))


def ep_skip_rms_norm_grad(dY, input_skip_bias_sum, gamma, inv_std_dev, dsum=None, dX=None, dgamma=True, dbias=None,
                          workspace=None, stream=None):
    """Gradient of the RMS norm, from the sum and the statistic that the forward
    call left (ep_skip_rms_norm_mx8, or ep_skip_layer_norm_ex in its simplified
    form).  ``dsum``: the gradient that reaches the sum along the residual stream.
    ``dgamma`` / ``dbias``: tensors to fill, True to allocate, or None.  Returns
    (dX, dgamma, dbias); dX is the gradient of input and of skip."""
    index, code = _first("dY", dY)
    other = _elsewhere(stream, index)
    if other is not None:
        with other:
            return ep_skip_rms_norm_grad(dY, input_skip_bias_sum, gamma, inv_std_dev, dsum, dX, dgamma, dbias, workspace)
    shape = dY.shape
    dims, rank, channels, _, stat_shape = _rows_plan(shape)
    _operand("input_skip_bias_sum", input_skip_bias_sum, dY, index, shape)
    _operand("gamma", gamma, dY, index, channels)
    if not isinstance(inv_std_dev, torch.Tensor):
        raise ValueError("inv_std_dev is required")
    _row_stats("inv_std_dev", inv_std_dev, dY, index, stat_shape)
    if dsum is not None:
        _operand("dsum", dsum, dY, index, shape)
    dX = torch.empty_like(dY) if dX is None else _operand("dX", dX, dY, index, shape)
    dgamma = _param_grad("dgamma", dgamma, dY, index, channels)
    dbias = _param_grad("dbias", dbias, dY, index, channels)
    s = _raw_stream(index)
    ws, wbytes, owned = _scratch(workspace, _rms_norm_grad_need(code, shape), dY, s)
    try:
        _check(load_library().ep_skip_rms_norm_grad(
            code, dY.data_ptr(), input_skip_bias_sum.data_ptr(), dims, rank, gamma.data_ptr(),
            inv_std_dev.data_ptr(), _addr(dsum), dX.data_ptr(), _addr(dgamma), _addr(dbias), ws, wbytes, s))
    finally:
        if owned:
            _raw_delete(ws)
    return dX, dgamma, dbias


@functools.lru_cache(maxsize=4096)
def _matmul_sizes(a_shape, w_shape):
    """(M, N, K), and the shapes of the result and of the bias, of A (..., K) times W (N, K)."""
    if len(a_shape) < 1 or len(w_shape) != 2 or a_shape[-1] != w_shape[1]:
        raise ValueError(f"A (..., K) and W (N, K) do not fit: {tuple(a_shape)} and {tuple(w_shape)}")
    shape, channels = torch.Size(a_shape[:-1] + w_shape[:1]), torch.Size(w_shape[:1])
    return torch.Size(a_shape[:-1]).numel(), w_shape[0], w_shape[1], shape, channels


@functools.lru_cache(maxsize=4096)
def _matmul_need(mx8, m, n, k, aligned):
    return int(load_library().ep_matmul_bias_act_workspace_size(int(mx8), m, n, k, int(aligned)))


@functools.lru_cache(maxsize=4096)
def _matmul_grad_need(m, n, k, activation, a_mx8, aligned):
    return int(load_library().ep_matmul_bias_act_grad_workspace_size(m, n, k, activation, int(a_mx8), int(aligned)))


def ep_matmul_bias_act_workspace_size(a_shape, w_shape, mx8=False, aligned=False) -> int:
    """Workspace bytes of ep_matmul_bias_act for A (..., K) and W (N, K), of 16 bits
    or (``mx8``) 8.  ``aligned``: both start on 16-byte boundaries."""
    m, n, k, _, _ = _matmul_sizes(torch.Size(a_shape), torch.Size(w_shape))
    return _matmul_need(bool(mx8), m, n, k, bool(aligned))


def ep_matmul_bias_act_grad_workspace_size(a_shape, w_shape, activation=EP_ACT_NONE, a_mx8=False, aligned=False) -> int:
    """Workspace bytes of ep_matmul_bias_act_grad.  ``a_mx8``: A is in MX8;
    ``aligned``: dY, W and a 16-bit A start on 16-byte boundaries."""
    m, n, k, _, _ = _matmul_sizes(torch.Size(a_shape), torch.Size(w_shape))
    return _matmul_grad_need(m, n, k, int(activation), bool(a_mx8), bool(aligned))


def ep_matmul_bias_act(A, W, bias=None, residual=None, activation=EP_ACT_NONE, alpha=DEFAULT_ALPHA, A_scales=None,
                       W_scales=None, dtype=None, Y=None, Z=None, Z_scales=None, workspace=None, stream=None):
    """Y = act(A W^T + bias) + residual for A (..., K) and W (N, K), both float16 or
    bfloat16, or both MX8 (float8_e4m3fn with ``A_scales`` and ``W_scales``; then
    ``dtype``, or the dtype of Y, residual or bias, is the result's).  ``Z``: the
    pre-activation, kept for the gradient: None, True (in the result's dtype),
    torch.float8_e4m3fn (in MX8), or a tensor to fill (with ``Z_scales`` if it is
    float8_e4m3fn).  Returns (Y, Z, Z_scales), the last two None when not requested."""
    if not isinstance(A, torch.Tensor) or not A.is_cuda:
        raise ValueError("A must be a CUDA tensor")
    index = A.get_device()
    other = _elsewhere(stream, index)
    if other is not None:
        with other:
            return ep_matmul_bias_act(A, W, bias, residual, activation, alpha, A_scales, W_scales, dtype, Y, Z,
                                      Z_scales, workspace)
    mx8 = A.dtype is _E4M3
    if not A.is_contiguous():
        raise ValueError("A must be contiguous")
    _operand("W", W, A, index)
    m, n, k, shape, channels = _matmul_sizes(A.shape, W.shape)
    if mx8:
        _operand("A_scales", A_scales, A, index, _scale_shape(A.shape), _E8M0)
        _operand("W_scales", W_scales, A, index, _scale_shape(W.shape), _E8M0)
        if dtype is None:
            like = Y if Y is not None else residual if residual is not None else bias
            if like is None:
                raise ValueError("dtype is required for 8-bit operands")
            dtype = like.dtype
    else:
        if A_scales is not None or W_scales is not None:
            raise ValueError("scales belong to float8_e4m3fn operands")
        if dtype is not None and dtype is not A.dtype:
            raise TypeError(f"dtype must be the operands' {A.dtype}, not {dtype}")
        dtype = A.dtype
    code = _TORCH_TO_EP.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    if bias is not None:
        _operand("bias", bias, A, index, channels, dtype)
    if residual is not None:
        _operand("residual", residual, A, index, shape, dtype)
    Y = torch.empty(shape, dtype=dtype, device=_cuda_device(index)) if Y is None else \
        _operand("Y", Y, A, index, shape, dtype)
    if Z is None and Z_scales is None:
        pass
    elif isinstance(Z, torch.dtype):
        if Z is not _E4M3 or Z_scales is not None:
            raise ValueError("Z: None, True, torch.float8_e4m3fn, or a tensor")
        Z, Z_scales = _mx8_out("Z", None, None, A, index, shape, _scale_shape(shape))
    elif isinstance(Z, torch.Tensor) and Z.dtype is _E4M3:
        if Z_scales is None:
            raise ValueError("Z_scales is required for a float8_e4m3fn Z")
        Z, Z_scales = _mx8_out("Z", Z, Z_scales, A, index, shape, _scale_shape(shape))
    else:
        if Z_scales is not None:
            raise ValueError("Z_scales belongs to a float8_e4m3fn Z")
        if Z is True:
            Z = torch.empty(shape, dtype=dtype, device=_cuda_device(index))
        elif Z is False:
            Z = None
        elif Z is not None:
            _operand("Z", Z, A, index, shape, dtype)
    lib = load_library()
    pa, pw = A.data_ptr(), W.data_ptr()
    s = _raw_stream(index)
    ws, wbytes, owned = _scratch(workspace, _matmul_need(mx8, m, n, k, (pa | pw) & 15 == 0), A, s)
    rest = (m, n, k, _addr(bias), _addr(residual), int(activation), float(alpha), Y.data_ptr(), _addr(Z),
            _addr(Z_scales), ws, wbytes, s)
    try:
        if mx8:
            _check(lib.ep_matmul_bias_act_mx8(code, pa, A_scales.data_ptr(), pw, W_scales.data_ptr(), *rest))
        else:
            _check(lib.ep_matmul_bias_act(code, pa, pw, *rest))
    finally:
        if owned:
            _raw_delete(ws)
    return Y, Z, Z_scales


def _grad_out(name, t, like, index, shape):
    if t is None or t is False:
        return None
    if t is True:
        return torch.empty(shape, dtype=like.dtype, device=_cuda_device(index))
    return _operand(name, t, like, index, shape)


def ep_matmul_bias_act_grad(dY, A, W, Z=None, activation=EP_ACT_NONE, alpha=DEFAULT_ALPHA, A_scales=None,
                            Z_scales=None, dA=True, dW=True, dbias=None, workspace=None, stream=None):
    """Gradient of ep_matmul_bias_act (the residual's is dY itself).  ``A`` and ``Z``
    (needed with an activation) are what the forward pass kept, each in dY's
    dtype or in MX8 (float8_e4m3fn with ``A_scales``, ``Z_scales``); ``W`` has dY's
    dtype.  ``dA`` / ``dW`` / ``dbias``: tensors to fill, True to allocate, or None.
    Returns (dA, dW, dbias), None where not requested."""
    index, code = _first("dY", dY)
    other = _elsewhere(stream, index)
    if other is not None:
        with other:
            return ep_matmul_bias_act_grad(dY, A, W, Z, activation, alpha, A_scales, Z_scales, dA, dW, dbias, workspace)
    _operand("W", W, dY, index)
    a_mx8 = A_scales is not None
    _operand("A", A, dY, index, dtype=_E4M3 if a_mx8 else None)
    m, n, k, shape, channels = _matmul_sizes(A.shape, W.shape)
    if a_mx8:
        _operand("A_scales", A_scales, dY, index, _scale_shape(A.shape), _E8M0)
    if dY.shape != shape:
        raise ValueError(f"dY must have shape {tuple(shape)}, not {tuple(dY.shape)}")
    activation = int(activation)
    if activation != EP_ACT_NONE:
        if Z is None:
            raise ValueError("Z is required with an activation")
        _operand("Z", Z, dY, index, shape, _E4M3 if Z_scales is not None else None)
        if Z_scales is not None:
            _operand("Z_scales", Z_scales, dY, index, _scale_shape(shape), _E8M0)
    dA = _grad_out("dA", dA, dY, index, A.shape)
    dW = _grad_out("dW", dW, dY, index, W.shape)
    dbias = _param_grad("dbias", dbias, dY, index, channels)
    py, pa, pw = dY.data_ptr(), A.data_ptr(), W.data_ptr()
    aligned = (py | pw | (0 if a_mx8 else pa)) & 15 == 0
    s = _raw_stream(index)
    ws, wbytes, owned = _scratch(workspace, _matmul_grad_need(m, n, k, activation, a_mx8, aligned), dY, s)
    try:
        _check(load_library().ep_matmul_bias_act_grad(
            code, py, pa, _addr(A_scales), pw, _addr(Z), _addr(Z_scales), m, n, k, activation, float(alpha), _addr(dA),
            _addr(dW), _addr(dbias), ws, wbytes, s))
    finally:
        if owned:
            _raw_delete(ws)
    return dA, dW, dbias
