"""The training and channels-last operators, as they are measured: group norm
with an optional SiLU (channels last) and its gradient, and bias + dropout +
residual, whose mask comes from a counter-based generator and is never stored,
and its gradient.

``run`` computes a case's operator either through the library (``own``) or in
its plain form: elementary torch operations in float32, rounded once at the
end.  ``exact`` is the definition in float64, written apart from both.
"""
import math

import numpy as np
import torch

own = False

EPSILON = 1e-5  # the GroupNorm contrib op's default

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}

# Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy
# as 1, 2, 3", SC 2011): the round multipliers and the key increments.
MULTIPLIERS = (0xD2511F53, 0xCD9E8D57)
INCREMENTS = (0x9E3779B9, 0xBB67AE85)
ROUNDS = 10
LOW = 0xFFFFFFFF


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _gn(name, op, n, s, c, groups, dtype, act):
    return dict(name=name, op=op, N=n, S=s, C=c, groups=groups, dtype=dtype, act=act)


def _drop(name, op, n, s, c, dtype, ratio, bias, residual=False):
    return dict(name=name, op=op, N=n, S=s, C=c, dtype=dtype, ratio=ratio, bias=bias, residual=residual)


def listed():
    return [
        # one decode step of eight sequences: the per-head norm of one token each
        _gn("gn token bf16 8x1x4096", "group_norm", 8, 1, 4096, 32, "bf16", "none"),
        # a channels-last block of a small batch, groups of 10 channels
        _gn("gn silu f16 2x4096x320", "group_norm", 2, 4096, 320, 32, "f16", "silu"),
        # odd sizes: rows that are no multiple of 16 bytes, 21 channels a group
        _gn("gn silu f16 3x1331x189", "group_norm", 3, 1331, 189, 9, "f16", "silu"),
        # a large channels-last batch: more data than the second-level cache holds
        _gn("gn silu bf16 8x16384x512", "group_norm", 8, 16384, 512, 32, "bf16", "silu"),
        # the gradient of an ordinary channels-last block
        _gn("gn grad silu f16 2x4096x640", "group_norm_grad", 2, 4096, 640, 32, "f16", "silu"),
        # the gradient of a per-head norm over the tokens of a training batch
        _gn("gn grad bf16 8192x1x2048", "group_norm_grad", 8192, 1, 2048, 16, "bf16", "none"),
        # a float32 gradient, ragged positions, groups of 12 channels
        _gn("gn grad silu f32 4x9999x384", "group_norm_grad", 4, 9999, 384, 32, "f32", "silu"),
        # the end of a block for a short sequence
        _drop("drop f16 1x128x1024", "bias_dropout", 1, 128, 1024, "f16", 0.1, True, True),
        # the end of a block over a training batch of tokens
        _drop("drop bf16 16x1024x4096", "bias_dropout", 16, 1024, 4096, "bf16", 0.1, True, True),
        # attention probabilities after the softmax: no bias, no residual
        _drop("drop f16 32x8192x512", "bias_dropout", 32, 8192, 512, "f16", 0.2, False),
        # the gradient over a training batch of tokens, with the bias's
        _drop("drop grad bf16 16x1024x4096", "bias_dropout_grad", 16, 1024, 4096, "bf16", 0.1, True),
        # float32 rows of odd length
        _drop("drop grad f32 3x1000x771", "bias_dropout_grad", 3, 1000, 771, "f32", 0.3, True),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["group_norm", "group_norm_grad", "bias_dropout", "bias_dropout_grad"])
    dtype = rng.choice(list(DTYPES))
    most = 1 << (25 if dtype == "f32" else 26)  # elements
    if op.startswith("group_norm"):
        most >>= op == "group_norm_grad"
        groups = rng.choice([1, 2, 3, 4, 8, 9, 16, 32, 32, 64])
        per_group = min(_log_int(rng, 1, 256), 8192 // groups)
        c = groups * per_group
        if rng.random() < 0.35:
            n, s = _log_int(rng, 1, 16384), rng.choice([1, 1, 1, 2, 5])  # tokens
        else:
            n, s = _log_int(rng, 1, 16), _log_int(rng, 1, 65536)  # positions of an image or a sequence
        s = max(-(-8 // per_group), min(s, most // (n * c)))  # a group has 8 values at least
        n = max(1, min(n, most // (s * c)))
        return dict(op=op, N=n, S=s, C=c, groups=groups, dtype=dtype, act=rng.choice(["none", "silu"]))
    c = _log_int(rng, 1, 8192)
    if rng.random() < 0.5:
        c = max(8, c // 8 * 8)
    s = min(_log_int(rng, 1, 65536), max(1, most // c))
    n = min(_log_int(rng, 1, 32), max(1, most // (s * c)))
    return dict(op=op, N=n, S=s, C=c, dtype=dtype, ratio=rng.choice([0.0, 0.05, 0.1, 0.2, 0.5, 0.9]),
                bias=rng.random() < 0.6, residual=op == "bias_dropout" and rng.random() < 0.6)


def work(case):
    e = case["N"] * case["S"] * case["C"]
    es, c = SIZES[case["dtype"]], case["C"]
    if case["op"] == "group_norm":
        stats = 2 * 4 * case["N"] * case["groups"]
        return dict(bytes=2 * e * es + 2 * c * es + stats, flops=e * (8 + 4 * (case["act"] == "silu")))
    if case["op"] == "group_norm_grad":
        stats = 2 * 4 * case["N"] * case["groups"]
        return dict(bytes=3 * e * es + 4 * c * es + stats, flops=e * (14 + 10 * (case["act"] == "silu")))
    if case["op"] == "bias_dropout":
        return dict(bytes=(2 + case["residual"]) * e * es + case["bias"] * c * es,
                    flops=e * (1 + case["bias"] + case["residual"]))
    return dict(bytes=2 * e * es + case["bias"] * c * es, flops=e * (1 + case["bias"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = DTYPES[case["dtype"]]
    shape = (case["N"], case["S"], case["C"])

    def normal(*dims, mean=0.0, std=1.0):
        return (torch.randn(*dims, device="cuda", generator=g) * std + mean).to(t)

    state = dict(case)
    if case["op"].startswith("group_norm"):
        # activations: channels of their own offset and spread around zero
        c = case["C"]
        spread = 0.5 + torch.rand(c, device="cuda", generator=g)
        centre = 0.3 + 0.5 * torch.randn(c, device="cuda", generator=g)
        state["X"] = (torch.randn(*shape, device="cuda", generator=g) * spread + centre).to(t)
        state["gamma"] = normal(c, mean=1.0, std=0.2)
        state["beta"] = normal(c, std=0.2)
        if case["op"] == "group_norm_grad":
            # what the forward pass left: float32 statistics
            x = state["X"].double().view(case["N"], case["S"], case["groups"], -1)
            m = x.mean((1, 3))
            v = ((x - m[:, None, :, None]) ** 2).mean((1, 3))
            state["mean"] = m.float()
            state["inv_std_dev"] = (1.0 / torch.sqrt(v + EPSILON)).float()
            state["dY"] = normal(*shape, std=0.5)
        return state
    state["seed"] = (seed * 0x9E3779B97F4A7C15 + 0x2545F4914F6CDD1D) % (1 << 62)
    state["offset"] = seed * 1000003 % (1 << 40)
    if case["op"] == "bias_dropout":
        state["X"] = normal(*shape)
        state["b"] = normal(case["C"], std=0.1) if case["bias"] else None
        state["R"] = normal(*shape) if case["residual"] else None
    else:
        state["dY"] = normal(*shape, std=0.5)
    return state


# ---------------------------------------------------------------------------
# the operators in their plain form
# ---------------------------------------------------------------------------

def _plain_group_norm(st):
    n, s, c, groups = st["N"], st["S"], st["C"], st["groups"]
    x = st["X"].float().view(n, s, groups, c // groups)
    mean = x.mean((1, 3))
    d = x - mean[:, None, :, None]
    inv = 1.0 / torch.sqrt((d * d).mean((1, 3)) + EPSILON)
    u = (d * inv[:, None, :, None]).view(n, s, c) * st["gamma"].float() + st["beta"].float()
    if st["act"] == "silu":
        u = u / (1.0 + torch.exp(-u))
    return u.to(st["X"].dtype), mean, inv


def _plain_group_norm_grad(st):
    n, s, c, groups = st["N"], st["S"], st["C"], st["groups"]
    t = st["X"].dtype
    gamma = st["gamma"].float()
    mean, inv = st["mean"][:, None, :, None], st["inv_std_dev"][:, None, :, None]
    h = ((st["X"].float().view(n, s, groups, c // groups) - mean) * inv).view(n, s, c)
    du = st["dY"].float()
    if st["act"] == "silu":
        u = h * gamma + st["beta"].float()
        sig = 1.0 / (1.0 + torch.exp(-u))
        du = du * (sig * (1.0 + u * (1.0 - sig)))
    dbeta = du.sum((0, 1))
    dgamma = (du * h).sum((0, 1))
    dh = (du * gamma).view(n, s, groups, c // groups)
    h = h.view(n, s, groups, c // groups)
    m1 = dh.mean((1, 3), keepdim=True)
    m2 = (dh * h).mean((1, 3), keepdim=True)
    dx = inv * (dh - m1 - h * m2)
    return dx.view(n, s, c).to(t), dgamma.to(t), dbeta.to(t)


def _plain_words(numel, seed, offset, device):
    """The generator's 32-bit words of elements 0..numel-1, as int64 (whose
    products wrap, so that the low and high halves of a 64-bit product are
    found by masking and shifting)."""
    block = torch.arange((numel + 3) // 4, device=device, dtype=torch.int64)
    c0, c1 = block & LOW, block >> 32
    c2, c3 = torch.full_like(block, offset & LOW), torch.full_like(block, offset >> 32)
    k0, k1 = seed & LOW, seed >> 32
    for _ in range(ROUNDS):
        p0, p1 = c0 * MULTIPLIERS[0], c2 * MULTIPLIERS[1]
        c0, c1, c2, c3 = ((p1 >> 32) & LOW) ^ c1 ^ k0, p1 & LOW, ((p0 >> 32) & LOW) ^ c3 ^ k1, p0 & LOW
        k0, k1 = (k0 + INCREMENTS[0]) & LOW, (k1 + INCREMENTS[1]) & LOW
    return torch.stack((c0, c1, c2, c3), 1).view(-1)[:numel]


def _plain_keep(st, shape):
    kept = round((1.0 - st["ratio"]) * 4294967296.0)
    return (_plain_words(math.prod(shape), st["seed"], st["offset"], "cuda") < kept).view(shape)


def _plain_bias_dropout(st):
    x = st["X"].float()
    if st["b"] is not None:
        x = x + st["b"].float()
    y = torch.where(_plain_keep(st, x.shape), x * (1.0 / (1.0 - st["ratio"])), 0.0)
    if st["R"] is not None:
        y = y + st["R"].float()
    return y.to(st["X"].dtype)


def _plain_bias_dropout_grad(st):
    dy = st["dY"].float()
    dx = torch.where(_plain_keep(st, dy.shape), dy * (1.0 / (1.0 - st["ratio"])), 0.0)
    dbias = dx.sum((0, 1)).to(st["dY"].dtype) if st["bias"] else None
    return dx.to(st["dY"].dtype), dbias


def run(state):
    op = state["op"]
    if own:
        import transformer_epilogue_gb300 as te

        act = te.EP_ACT_SILU if state.get("act") == "silu" else te.EP_ACT_NONE
        if op == "group_norm":
            return te.ep_group_norm(state["X"], state["gamma"], state["beta"], groups=state["groups"],
                                    epsilon=EPSILON, activation=act, mean=True, inv_std_dev=True)
        if op == "group_norm_grad":
            return te.ep_group_norm_grad(state["dY"], state["X"], state["gamma"], state["beta"],
                                         state["mean"], state["inv_std_dev"], groups=state["groups"],
                                         activation=act)
        if op == "bias_dropout":
            return te.ep_bias_dropout(state["X"], state["ratio"], state["seed"], state["offset"],
                                      bias=state["b"], residual=state["R"])
        return te.ep_bias_dropout_grad(state["dY"], state["ratio"], state["seed"], state["offset"],
                                       dbias=True if state["bias"] else None)
    if op == "group_norm":
        return _plain_group_norm(state)
    if op == "group_norm_grad":
        return _plain_group_norm_grad(state)
    if op == "bias_dropout":
        return _plain_bias_dropout(state)
    return _plain_bias_dropout_grad(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _sample_stats(x, groups):
    """Mean and 1/sqrt(variance + epsilon) of each group of one sample (S, C)."""
    by_group = x.reshape(x.shape[0], groups, -1).transpose(0, 1).reshape(groups, -1)
    mean = by_group.sum(1) / by_group.shape[1]
    var = ((by_group - mean[:, None]) ** 2).sum(1) / by_group.shape[1]
    return mean, (var + EPSILON) ** -0.5


def _exact_group_norm(st):
    per = st["C"] // st["groups"]
    gamma, beta = st["gamma"].double(), st["beta"].double()
    if st["S"] <= 8:  # many tokens: all samples at once, each group a row
        x = st["X"].double().view(st["N"], st["S"], st["groups"], per).permute(0, 2, 1, 3)
        flat = x.reshape(st["N"], st["groups"], -1)
        mean = flat.sum(2) / flat.shape[2]
        inv = (((flat - mean[..., None]) ** 2).sum(2) / flat.shape[2] + EPSILON) ** -0.5
        u = ((x - mean[..., None, None]) * inv[..., None, None]).permute(0, 2, 1, 3)
        u = u.reshape(st["N"], st["S"], st["C"]) * gamma + beta
        return (u * torch.sigmoid(u) if st["act"] == "silu" else u), mean, inv
    out, means, invs = [], [], []
    for sample in st["X"]:
        x = sample.double()
        mean, inv = _sample_stats(x, st["groups"])
        u = (x - mean.repeat_interleave(per)) * (inv.repeat_interleave(per) * gamma) + beta
        out.append(u * torch.sigmoid(u) if st["act"] == "silu" else u)
        means.append(mean)
        invs.append(inv)
    return torch.stack(out), torch.stack(means), torch.stack(invs)


def _exact_group_norm_grad(st):
    n, groups = st["N"], st["groups"]
    per = st["C"] // groups
    count = st["S"] * per
    gamma, beta = st["gamma"].double(), st["beta"].double()
    mean = st["mean"].double().repeat_interleave(per, 1)
    inv = st["inv_std_dev"].double().repeat_interleave(per, 1)
    dx = torch.empty(st["X"].shape, dtype=torch.float64, device="cuda")
    dgamma, dbeta = torch.zeros_like(gamma), torch.zeros_like(beta)
    step = max(1, (1 << 22) // (st["S"] * st["C"]))
    for i in range(0, n, step):
        h = (st["X"][i:i + step].double() - mean[i:i + step, None]) * inv[i:i + step, None]
        du = st["dY"][i:i + step].double()
        if st["act"] == "silu":
            u = h * gamma + beta
            sig = torch.sigmoid(u)
            du = du * (sig + u * sig * (1.0 - sig))
        sums = du.sum(1)      # per sample and channel
        sums_h = (du * h).sum(1)
        dbeta += sums.sum(0)
        dgamma += sums_h.sum(0)
        m1 = (sums * gamma).view(-1, groups, per).sum(2) / count
        m2 = (sums_h * gamma).view(-1, groups, per).sum(2) / count
        dx[i:i + step] = inv[i:i + step, None] * (du * gamma - m1.repeat_interleave(per, 1)[:, None]
                                                  - h * m2.repeat_interleave(per, 1)[:, None])
    return dx, dgamma, dbeta


def _exact_keep(st):
    """The mask from unsigned 64-bit host arithmetic."""
    numel = st["N"] * st["S"] * st["C"]
    blocks = -(-numel // 4)
    words = np.empty((blocks, 4), dtype=np.uint32)
    chunk = 1 << 20
    half = np.uint64(32)
    low = np.uint64(LOW)
    for at in range(0, blocks, chunk):
        i = np.arange(at, min(at + chunk, blocks), dtype=np.uint64)
        x = [i & low, i >> half, np.full_like(i, st["offset"] & LOW), np.full_like(i, st["offset"] >> 32)]
        key = [st["seed"] & LOW, st["seed"] >> 32]
        for _ in range(ROUNDS):
            a, b = np.uint64(MULTIPLIERS[0]) * x[0], np.uint64(MULTIPLIERS[1]) * x[2]
            x = [(b >> half) ^ x[1] ^ np.uint64(key[0]), b & low, (a >> half) ^ x[3] ^ np.uint64(key[1]), a & low]
            key = [(key[0] + INCREMENTS[0]) % (1 << 32), (key[1] + INCREMENTS[1]) % (1 << 32)]
        for w in range(4):
            words[at:at + chunk, w] = x[w]
    kept = int(round((1.0 - st["ratio"]) * 2.0 ** 32))
    keep = words.reshape(-1)[:numel].astype(np.uint64) < np.uint64(kept)
    return torch.from_numpy(keep).view(st["N"], st["S"], st["C"]).cuda()


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "group_norm":
        return _exact_group_norm(st)
    if case["op"] == "group_norm_grad":
        return _exact_group_norm_grad(st)
    keep = _exact_keep(st).double()
    if case["op"] == "bias_dropout":
        x = st["X"].double()
        if st["b"] is not None:
            x = x + st["b"].double()
        y = x * keep / (1.0 - case["ratio"])
        return y if st["R"] is None else y + st["R"].double()
    dx = st["dY"].double() * keep / (1.0 - case["ratio"])
    return dx, (dx.sum((0, 1)) if case["bias"] else None)
