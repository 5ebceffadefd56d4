"""The 8-bit and matrix operators, as they are measured: the root-mean-square
norm with the residual's addition and an 8-bit output, its gradient, rows held
in 8 bits, and the matrix product with bias, activation and residual in its
epilogue (of 16-bit and of 8-bit operands) with its gradient, which reads what
the forward pass left in 16 or in 8 bits.

8 bits are MX8 (the OCP microscaling format MXFP8 with E4M3 elements): 32
consecutive elements of a row share one power-of-two scale, the smallest that
brings the largest of them within 448.

``run`` computes a case's operator either through the library (``own``) or in
its plain form: elementary torch operations in float32, rounded once at the
end.  ``exact`` is the definition in float64, written apart from both.
"""
import math

import torch

own = False

EPSILON = 9.999999960041972e-13  # SkipLayerNormalization's default
ALPHA = 1.702                    # QuickGelu's default
GROUP = 32                       # elements that share a scale
E4M3_MOST = 448.0

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
ACTS = ("none", "silu", "relu", "quick_gelu", "gelu", "fast_gelu")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(name, op, m, h, dtype, extra):
    # extra: the bias before the norm (and its gradient)
    return dict(name=name, op=op, M=m, H=h, dtype=dtype, extra=extra)


def _mm(name, op, m, k, n, dtype, act, bias=True, residual=False, save="none", kept="t"):
    # save: how the forward pass keeps the pre-activation ("none", "t", "mx8");
    # kept: how the gradient finds the product's left operand ("t", "mx8")
    return dict(name=name, op=op, M=m, K=k, N=n, dtype=dtype, act=act, bias=bias, residual=residual, save=save,
                kept=kept)


def listed():
    return [
        # one decode step of eight sequences: residual added, normed, ready for an 8-bit product
        _norm("norm mx8 bf16 8x4096", "norm_mx8", 8, 4096, "bf16", False),
        # a training batch of tokens (the norm's benchmark shape)
        _norm("norm mx8 bf16 16384x4096", "norm_mx8", 16384, 4096, "bf16", True),
        # its gradient over the same batch
        _norm("norm grad bf16 16384x4096", "norm_grad", 16384, 4096, "bf16", False),
        # float32 rows of odd length and odd count, with the bias's gradient
        _norm("norm grad f32 2053x1001", "norm_grad", 2053, 1001, "f32", True),
        # an activation of a long batch put aside in 8 bits
        _norm("quantize f16 8192x4096", "quantize", 8192, 4096, "f16", False),
        # one decode step of eight sequences through the first layer of a feed-forward block
        _mm("mm bf16 8x4096x16384", "matmul", 8, 4096, 16384, "bf16", "quick_gelu"),
        # odd sizes throughout, with a residual
        _mm("mm f16 1331x771x1001", "matmul", 1331, 771, 1001, "f16", "gelu", residual=True),
        # a training batch through the first layer of a feed-forward block, the pre-activation kept
        _mm("mm save bf16 8192x4096x16384", "matmul", 8192, 4096, 16384, "bf16", "quick_gelu", save="t"),
        # one decode step of sixteen sequences through 8-bit weights, added to the residual stream
        _mm("mm mx8 bf16 16x4096x4096", "matmul_mx8", 16, 4096, 4096, "bf16", "none", residual=True),
        # a training batch through 8-bit weights, the pre-activation kept in 8 bits
        _mm("mm mx8 save8 bf16 8192x4096x8192", "matmul_mx8", 8192, 4096, 8192, "bf16", "fast_gelu", save="mx8"),
        # the gradient of an ordinary first layer: everything kept in 16 bits
        _mm("mm grad bf16 4096x1024x4096", "matmul_grad", 4096, 1024, 4096, "bf16", "quick_gelu", save="t"),
        # the gradient of a large one from 8-bit checkpoints of its input and its pre-activation
        _mm("mm grad8 bf16 8192x4096x4096", "matmul_grad", 8192, 4096, 4096, "bf16", "fast_gelu", save="mx8",
            kept="mx8"),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _size(rng, low, high):
    """Sizes over [low, high]: half of them multiples of 64, as layers have, the others any."""
    v = _log_int(rng, low, high)
    return max(64, v // 64 * 64) if rng.random() < 0.5 and high >= 64 else v


def draw(rng):
    op = rng.choice(["norm_mx8", "norm_grad", "quantize", "matmul", "matmul", "matmul_mx8", "matmul_grad"])
    if op in ("norm_mx8", "norm_grad", "quantize"):
        dtype = rng.choice(list(DTYPES))
        h = _size(rng, 1, 16384)
        most = 1 << (25 if dtype == "f32" else 26)
        m = max(-(-64 // h), min(_log_int(rng, 1, 65536), most // h))  # a few values at least
        return dict(op=op, M=m, H=h, dtype=dtype, extra=rng.random() < 0.5)
    dtype = rng.choice(["f16", "bf16"])
    k, n = _size(rng, 1, 16384), _size(rng, 1, 16384)
    most = 1 << (38 if op != "matmul_grad" else 36)  # products of two numbers
    m = _log_int(rng, 1, 256) if rng.random() < 0.4 else _log_int(rng, 1, 16384)
    m = max(-(-16 // n), min(m, most // (k * n), (1 << 26) // max(k, n)))
    if op == "matmul_grad":
        act = rng.choice(ACTS)
        save = rng.choice(["t", "mx8"]) if act != "none" else "none"
        return dict(op=op, M=m, K=k, N=n, dtype=dtype, act=act, bias=rng.random() < 0.7, residual=False, save=save,
                    kept=rng.choice(["t", "mx8"]))
    return dict(op=op, M=m, K=k, N=n, dtype=dtype, act=rng.choice(ACTS), bias=rng.random() < 0.7,
                residual=rng.random() < 0.5, save=rng.choice(["none", "none", "t", "mx8"]), kept="t")


def _groups(n):
    return -(-n // GROUP)


def _held(rows, cols, how, es):
    """Bytes of a (rows, cols) array held in T or in 8 bits with scales."""
    return {"none": 0, "t": rows * cols * es, "mx8": rows * (cols + _groups(cols))}[how]


def work(case):
    es, m = SIZES[case["dtype"]], case["M"]
    if case["op"] in ("norm_mx8", "norm_grad", "quantize"):
        h = case["H"]
        q = _held(m, h, "mx8", es)
        if case["op"] == "quantize":
            return dict(bytes=m * h * es + q, flops=3 * m * h)
        if case["op"] == "norm_mx8":  # input, skip and their sum, gamma, the bias, the statistic
            return dict(bytes=3 * m * h * es + q + (1 + case["extra"]) * h * es + 4 * m, flops=8 * m * h)
        # dY, the sum, the gradient that comes along the residual, and dX; gamma and the parameters' gradients
        return dict(bytes=4 * m * h * es + (2 + case["extra"]) * h * es + 4 * m, flops=10 * m * h)
    k, n = case["K"], case["N"]
    if case["op"] == "matmul_grad":
        return dict(bytes=m * n * es + _held(m, n, case["save"], es) + _held(m, k, case["kept"], es) + n * k * es
                    + m * k * es + n * k * es + case["bias"] * n * es, flops=4 * m * n * k)
    how = "mx8" if case["op"] == "matmul_mx8" else "t"
    return dict(bytes=_held(m, k, how, es) + _held(n, k, how, es) + (1 + case["residual"]) * m * n * es
                + _held(m, n, case["save"], es) + case["bias"] * n * es, flops=2 * m * n * k)


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

def _padded(x):
    """The groups of a (rows, cols) array: (rows, groups, 32), zeros behind the last column."""
    rows, cols = x.shape
    return torch.nn.functional.pad(x, (0, _groups(cols) * GROUP - cols)).view(rows, -1, GROUP)


def _quantize(x):
    """float32 (rows, cols) -> E4M3 elements and power-of-two scales.  2^(127-b) * amax <= 448 < 2^(128-b) * amax."""
    g = _padded(x)
    frac, exp = torch.frexp(g.abs().amax(2))            # amax = frac * 2^exp, frac in [0.5, 1)
    byte = (exp - 9 + (frac > E4M3_MOST / 512) + 127).clamp(1, 254)
    q = torch.ldexp(g, 127 - byte[..., None]).clamp(-E4M3_MOST, E4M3_MOST)
    q = q.view(x.shape[0], -1)[:, : x.shape[1]].contiguous().to(torch.float8_e4m3fn)
    return q, byte.to(torch.uint8).view(torch.float8_e8m0fnu)


def _dequantize(q, scales):
    byte = scales.view(torch.uint8).int()
    return torch.ldexp(_padded(q.float()), byte[..., None] - 127).view(q.shape[0], -1)[:, : q.shape[1]]


def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "relu":
        return torch.relu(z)
    if act == "quick_gelu":
        return z * torch.sigmoid(ALPHA * z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "fast_gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act in ("silu", "quick_gelu"):
        a = 1.0 if act == "silu" else ALPHA
        s = torch.sigmoid(a * z)
        return s + a * z * s * (1 - s)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "fast_gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain(s):
    t = DTYPES[s["dtype"]]
    if s["op"] == "quantize":
        return dict(zip(("q", "scales"), _quantize(s["X"].float())))
    if s["op"] == "norm_mx8":
        v = s["X"].float() + s["skip"].float()
        if s["extra"]:
            v = v + s["b"].float()
        inv = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPSILON)
        q, scales = _quantize(v * inv * s["gamma"].float())
        return dict(q=q, scales=scales, sum=v.to(t), inv=inv)
    if s["op"] == "norm_grad":
        v, dy, inv = s["S"].float(), s["dY"].float(), s["inv"]
        x = v * inv
        u = dy * s["gamma"].float()
        dx = inv * (u - x * (u * x).mean(1, keepdim=True)) + s["dS"].float()
        out = dict(dX=dx.to(t), dgamma=(dy * x).sum(0).to(t))
        if s["extra"]:
            out["dbias"] = dx.sum(0).to(t)
        return out
    if s["op"] == "matmul_grad":
        dz = s["dY"].float()
        if s["act"] != "none":
            z = s["Z"].float() if s["save"] == "t" else _dequantize(s["Z"], s["Zs"])
            dz = dz * _act_grad(z, s["act"])
        a = s["A"].float() if s["kept"] == "t" else _dequantize(s["A"], s["As"])
        out = dict(dA=(dz @ s["W"].float()).to(t), dW=(dz.t() @ a).to(t))
        if s["bias"]:
            out["dbias"] = dz.sum(0).to(t)
        return out
    if s["op"] == "matmul_mx8":
        z = _dequantize(s["A"], s["As"]) @ _dequantize(s["W"], s["Ws"]).t()
    else:
        z = s["A"].float() @ s["W"].float().t()
    if s["bias"]:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["residual"]:
        y = y + s["R"].float()
    out = dict(y=y.to(t))
    if s["save"] == "t":
        out["z"] = z.to(t)
    elif s["save"] == "mx8":
        out["z"], out["z_scales"] = _quantize(z)
    return out


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own(s):
    import transformer_epilogue_gb300 as te
    if s["op"] == "quantize":
        return dict(zip(("q", "scales"), te.ep_quantize_mx8(s["X"])))
    if s["op"] == "norm_mx8":
        return dict(zip(("q", "scales", "sum", "inv"), te.ep_skip_rms_norm_mx8(
            s["X"], s["skip"], s["gamma"], bias=s.get("b"), input_skip_bias_sum=True, inv_std_dev=True)))
    if s["op"] == "norm_grad":
        dx, dg, db = te.ep_skip_rms_norm_grad(s["dY"], s["S"], s["gamma"], s["inv"], dsum=s["dS"],
                                              dbias=True if s["extra"] else None)
        return dict(dX=dx, dgamma=dg, dbias=db) if s["extra"] else dict(dX=dx, dgamma=dg)
    act = dict(none=te.EP_ACT_NONE, silu=te.EP_ACT_SILU, relu=te.EP_ACT_RELU, quick_gelu=te.EP_ACT_QUICK_GELU,
               gelu=te.EP_ACT_GELU, fast_gelu=te.EP_ACT_FAST_GELU)[s["act"]]
    if s["op"] == "matmul_grad":
        da, dw, db = te.ep_matmul_bias_act_grad(
            s["dY"], s["A"], s["W"], Z=s.get("Z"), activation=act, alpha=ALPHA, A_scales=s.get("As"),
            Z_scales=s.get("Zs"), dbias=True if s["bias"] else None)
        return dict(dA=da, dW=dw, dbias=db) if s["bias"] else dict(dA=da, dW=dw)
    save = {"none": None, "t": True, "mx8": torch.float8_e4m3fn}[s["save"]]
    y, z, zs = te.ep_matmul_bias_act(
        s["A"], s["W"], bias=s.get("b"), residual=s.get("R"), activation=act, alpha=ALPHA, A_scales=s.get("As"),
        W_scales=s.get("Ws"), dtype=DTYPES[s["dtype"]], Z=save)
    out = dict(y=y)
    if z is not None:
        out["z"] = z
    if zs is not None:
        out["z_scales"] = zs
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = DTYPES[case["dtype"]]

    def normal(*dims, mean=0.0, std=1.0):
        return (torch.randn(*dims, device="cuda", generator=g) * std + mean).to(t)

    def activations(rows, cols):
        """A residual stream: one channel in fifty is several times as wide as the others."""
        wide = torch.rand(cols, device="cuda", generator=g) < 0.02
        return (torch.randn(rows, cols, device="cuda", generator=g) * (1 + 7 * wide)).to(t)

    state, m = dict(case), case["M"]
    if case["op"] in ("norm_mx8", "norm_grad", "quantize"):
        h = case["H"]
        state["X"] = activations(m, h)
        if case["op"] == "quantize":
            return state
        state["gamma"] = normal(h, mean=1.0, std=0.2)
        if case["op"] == "norm_mx8":
            state["skip"] = normal(m, h, std=0.5)
            if case["extra"]:
                state["b"] = normal(h, std=0.1)
            return state
        # what the forward pass left
        state["S"] = state.pop("X")
        v = state["S"].double()
        state["inv"] = (1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPSILON)).float()
        state["dY"] = normal(m, h, std=0.5)
        state["dS"] = normal(m, h, std=0.5)
        return state
    k, n = case["K"], case["N"]
    a, w = normal(m, k), normal(n, k, std=1 / math.sqrt(k))
    b = normal(n, std=0.1)
    if case["bias"]:
        state["b"] = b
    if case["op"] == "matmul_grad":
        if case["save"] != "none":
            z = a.float() @ w.float().t() + b.float()
            if case["save"] == "t":
                state["Z"] = z.to(t)
            else:
                state["Z"], state["Zs"] = _quantize(z)
        state["dY"] = normal(m, n, std=0.5)
    elif case["residual"]:
        state["R"] = normal(m, n)
    state["A"], state["W"] = a, w
    if case["op"] == "matmul_mx8" or case["kept"] == "mx8":
        state["A"], state["As"] = _quantize(a.float())
    if case["op"] == "matmul_mx8":
        state["W"], state["Ws"] = _quantize(w.float())
    return state


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_scaled(v):
    """v / scale, before it is rounded to 8 bits: the scale of 32 neighbours is the smallest power of two >= amax / 448."""
    rows, cols = v.shape
    out = torch.empty_like(v)
    whole = cols // GROUP * GROUP
    for part in (slice(0, whole), slice(whole, cols)):
        p = v[:, part]
        if p.shape[1] == 0:
            continue
        p = p.reshape(rows, -1, min(GROUP, p.shape[1]))
        e = torch.ceil(torch.log2(p.abs().max(2, keepdim=True).values / E4M3_MOST)).clamp(min=-126)
        out[:, part] = (p * torch.exp2(-e)).reshape(rows, -1)
    return out


def _value(q, scales):
    """What 8 bits with scales stand for."""
    s = torch.exp2(scales.view(torch.uint8).double() - 127)
    return q.double() * s.repeat_interleave(GROUP, 1)[:, : q.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items()
         if isinstance(v, torch.Tensor) and v.dtype in (torch.float32, torch.float16, torch.bfloat16)}
    if case["op"] == "quantize":
        return dict(q=_exact_scaled(d["X"]), scales=None)
    if case["op"] == "norm_mx8":
        v = d["X"] + d["skip"]
        if case["extra"]:
            v += d["b"]
        inv = torch.rsqrt(v.square().sum(1) / case["H"] + EPSILON)[:, None]
        # (the scales have no value of their own here: a maximum next to a power of two may fall on either side)
        return dict(q=_exact_scaled(v * inv * d["gamma"]), scales=None, sum=v, inv=inv)
    if case["op"] == "norm_grad":
        # the derivative of v_j / sqrt(mean(v^2) + eps) by v_i is inv (delta_ij - v_i v_j inv^2 / H)
        v, inv, u = d["S"], d["inv"], d["dY"] * d["gamma"]
        dx = inv * u - v * inv ** 3 * (u * v).sum(1, keepdim=True) / case["H"] + d["dS"]
        out = dict(dX=dx, dgamma=torch.einsum("mh,mh->h", d["dY"], v * inv))
        if case["extra"]:
            out["dbias"] = dx.sum(0)
        return out

    def derivative(z):
        """(activation, its derivative) at z."""
        if case["act"] == "none":
            return z, torch.ones_like(z)
        if case["act"] == "relu":
            return z.clamp(min=0), torch.where(z > 0, 1.0, 0.0).double()
        if case["act"] == "gelu":
            cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2))
            return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        if case["act"] == "fast_gelu":  # (1 + tanh(x)) / 2 = 1 / (1 + exp(-2 x))
            x = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
            slope = 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2)
        else:
            slope = 1.0 if case["act"] == "silu" else ALPHA
            x = slope * z
        p = 1 / (1 + torch.exp(-x))
        return z * p, p + z * slope * p / (1 + torch.exp(x))

    a = _value(s["A"], s["As"]) if "As" in s else d["A"]
    if case["op"] == "matmul_grad":
        dz = d["dY"]
        if case["act"] != "none":
            dz = dz * derivative(_value(s["Z"], s["Zs"]) if "Zs" in s else d["Z"])[1]
        out = dict(dA=dz.matmul(d["W"]), dW=dz.t().matmul(a))
        if case["bias"]:
            out["dbias"] = dz.sum(0)
        return out
    w = _value(s["W"], s["Ws"]) if "Ws" in s else d["W"]
    z = torch.matmul(a, w.t())
    if case["bias"]:
        z += d["b"]
    y = derivative(z)[0]
    out = dict(y=y + d["R"] if case["residual"] else y)
    if case["save"] == "t":
        out["z"] = z
    elif case["save"] == "mx8":
        out.update(z=_exact_scaled(z), z_scales=None)
    return out
