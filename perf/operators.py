"""What is measured of the residual branch's operators, with their plain forms.

A residual branch x + dropout(f(layernorm(x))) around a gated pointwise block is what a
training program runs next to this package's convolution gradients: layer norm over the
channels of NHWC rows, the gated pointwise block h = act(g) * u with [g | u] = x W^T, and
dropout from a counter-based generator, each with its backward pass.

``listed()`` names the cases, ``draw(rng)`` makes more of the same ranges, ``prepare`` makes
the inputs, ``run`` makes one pass (the plain form, or the package's calls when ``own`` is
set), ``work`` counts what the pass cannot do without and ``exact`` evaluates the
definition in 64 bits.

Definitions (rows m, channels c, all over the last axis):
  layer norm   mean = sum(x)/C, rstd = 1/sqrt(sum((x-mean)^2)/C + eps),
               y = (x - mean)*rstd*gamma + beta; backward, with n = (x-mean)*rstd and
               q = dy*gamma: dx = rstd*(q - mean_c(q) - n*mean_c(q*n)),
               dgamma = sum_m dy*n, dbeta = sum_m dy.
  gated        z = [g | u] = x W^T with W (2F, C), h = act(g)*u; backward from dh, x, z, W:
               dg = dh*u*act'(g), du = dh*act(g), dx = [dg | du] W, dW = [dg | du]^T x.
  dropout      element i belongs to block b = i // 8 and takes 16 bits of Philox-4x32-10
               (J. Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011) at
               counter (b, offset) and key seed: word (i % 8) // 2, its low half for even i.
               With t = round(p * 65536) the element is kept where its draw is >= t, and then
               is scaled by 65536/(65536 - t); y = kept x (+ residual).
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


def listed():
    return [
        # one decoding step of a few sequences: latency
        {"name": "ln_fwd_token", "op": "ln_fwd", "dtype": "bf16", "M": 4, "C": 768, "stats": False},
        # the 64x64 stage of a convolutional network, batch 16, training: 384 channels
        {"name": "ln_fwd_stage", "op": "ln_fwd", "dtype": "bf16", "M": 16 * 64 * 64, "C": 384, "stats": True},
        # ragged rows of odd length in full precision
        {"name": "ln_bwd_odd", "op": "ln_bwd", "dtype": "f32", "M": 37 * 53, "C": 1001},
        # the early 112x112 stage, batch 32: many short rows
        {"name": "ln_bwd_early", "op": "ln_bwd", "dtype": "bf16", "M": 32 * 112 * 112, "C": 96},
        # one token through the block: the weights' bytes and latency
        {"name": "gated_fwd_token", "op": "gated_fwd", "dtype": "bf16", "M": 1, "C": 768, "F": 2048,
         "act": "silu", "keep": False},
        # a ragged prompt with odd tile tails
        {"name": "gated_fwd_ragged", "op": "gated_fwd", "dtype": "f16", "M": 37 * 53, "C": 328, "F": 1000,
         "act": "gelu", "keep": False},
        # a training forward at 768 channels, 8 images of 64x64, pre-activations kept
        {"name": "gated_fwd_train", "op": "gated_fwd", "dtype": "bf16", "M": 8 * 64 * 64, "C": 768, "F": 2048,
         "act": "silu", "keep": True},
        # the benchmark's pointwise rows (8 images of 56x56) with a small block: long sums in dW, few tiles
        {"name": "gated_bwd_stage", "op": "gated_bwd", "dtype": "bf16", "M": 8 * 56 * 56, "C": 256, "F": 512,
         "act": "silu"},
        # a language model's block, 16384 tokens
        {"name": "gated_bwd_wide", "op": "gated_bwd", "dtype": "f16", "M": 16384, "C": 1024, "F": 4096,
         "act": "gelu_tanh"},
        # residual branch at the 64x64 stage
        {"name": "drop_fwd_residual", "op": "drop_fwd", "dtype": "bf16", "M": 16 * 64 * 64, "C": 384, "p": 0.1,
         "residual": True},
        # ragged and odd, in full precision
        {"name": "drop_bwd_odd", "op": "drop_bwd", "dtype": "f32", "M": 37 * 53, "C": 1001, "p": 0.5},
        # the early stage's gradients
        {"name": "drop_bwd_early", "op": "drop_bwd", "dtype": "f16", "M": 32 * 112 * 112, "C": 96, "p": 0.2},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "gated_fwd", "gated_bwd", "drop_fwd", "drop_bwd"])
    if op.startswith("gated"):
        # channels are whole 16-byte rows
        C = 8 * _log(rng, 8, 256)
        F = 8 * _log(rng, 8, 700)
        most = 2.5e11 if op == "gated_bwd" else 1.5e11
        M = _log(rng, 1, max(1, min(32768, int(most / (4 * C * F)))))
        case = {"op": op, "dtype": rng.choice(["bf16", "f16"]), "M": M, "C": C, "F": F,
                "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])}
        if op == "gated_fwd":
            case["keep"] = rng.random() < 0.5
        return case
    C = _log(rng, 8, 12288)
    M = _log(rng, 1, max(1, 30_000_000 // C))
    case = {"op": op, "dtype": rng.choice(["f32", "bf16", "f16"]), "M": M, "C": C}
    if op == "ln_fwd":
        case["stats"] = rng.random() < 0.5
    if op.startswith("drop"):
        case["p"] = round(rng.uniform(0.01, 0.6), 4)
    if op == "drop_fwd":
        case["residual"] = rng.random() < 0.5
    return case


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = _TYPES[case["dtype"]]
    M, C, op = case["M"], case["C"], case["op"]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device="cuda") * std + mean

    s = dict(case)
    if op.startswith("ln"):
        # activations: a common offset, channels of unlike scale
        scale = normal(C, std=0.4).exp()
        s["x"] = (normal(M, C) * scale + normal(C, std=0.5)).to(t)
        s["gamma"] = normal(C, std=0.2, mean=1.0).to(t)
        if op == "ln_fwd":
            s["beta"] = normal(C, std=0.2).to(t)
        else:
            s["dy"] = normal(M, C, std=0.3).to(t)
            xf = s["x"].float()
            s["mean"] = xf.sum(1) / C
            s["rstd"] = 1.0 / torch.sqrt(((xf - s["mean"][:, None]) ** 2).sum(1) / C + EPS)
    elif op.startswith("gated"):
        F = case["F"]
        s["x"] = normal(M, C).to(t)
        s["w"] = normal(2 * F, C, std=C ** -0.5).to(t)
        if op == "gated_bwd":
            s["dh"] = normal(M, F, std=0.2).to(t)
            s["z"] = (s["x"].float() @ s["w"].float().T).to(t)
    else:
        s["x"] = normal(M, C).to(t)
        if case.get("residual"):
            s["r"] = normal(M, C, std=2.0).to(t)
        s["seed"] = 0x9E3779B97F4A7C15 * (seed + 1) & (2 ** 64 - 1)
        s["offset"] = 3 + (seed << 33)
    return s


# ------------------------------------------------------------------ plain forms

def _act(name, g):
    """act(g) and act'(g)."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if name == "sigmoid":
        s = 1 / (1 + torch.exp(-g))
        return s, s * (1 - s)
    if name == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(g * (0.5 ** 0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    k = math.sqrt(2 / math.pi)
    th = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * k * (1 + 3 * 0.044715 * g * g)


def _mulhilo(a, const):
    """High and low 32 bits of a * const for 32-bit values held in int64."""
    lo_p = (a & 0xFFFF) * const
    hi_p = (a >> 16) * const
    mid = hi_p + (lo_p >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (lo_p & 0xFFFF)


def _keep(n, p, seed, offset, device):
    """Truth values of n elements' draws and the scale of what is kept."""
    b = torch.arange((n + 7) // 8, device=device, dtype=torch.int64)
    c0, c1 = b & 0xFFFFFFFF, b >> 32
    c2 = torch.full_like(b, offset & 0xFFFFFFFF)
    c3 = torch.full_like(b, offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    t = int(round(p * 65536))
    draws = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF,
                         c3 >> 16], 1).reshape(-1)[:n]
    return draws >= t, 65536.0 / (65536 - t)


def _plain(s):
    op = s["op"]
    t = s["x"].dtype
    x = s["x"].float()
    C = s["C"]
    if op == "ln_fwd":
        mean = x.sum(1, keepdim=True) / C
        d = x - mean
        rstd = 1.0 / torch.sqrt((d * d).sum(1, keepdim=True) / C + EPS)
        y = (d * rstd * s["gamma"].float() + s["beta"].float()).to(t)
        return (y, mean[:, 0], rstd[:, 0]) if s["stats"] else (y,)
    if op == "ln_bwd":
        dy = s["dy"].float()
        rstd = s["rstd"][:, None]
        n = (x - s["mean"][:, None]) * rstd
        q = dy * s["gamma"].float()
        dx = rstd * (q - q.sum(1, keepdim=True) / C - n * ((q * n).sum(1, keepdim=True) / C))
        return dx.to(t), (dy * n).sum(0).to(t), dy.sum(0).to(t)
    if op == "gated_fwd":
        z = x @ s["w"].float().T
        F = s["F"]
        h = (_act(s["act"], z[:, :F])[0] * z[:, F:]).to(t)
        return (h, z.to(t)) if s["keep"] else (h,)
    if op == "gated_bwd":
        F = s["F"]
        z = s["z"].float()
        dh = s["dh"].float()
        a, da = _act(s["act"], z[:, :F])
        dz = torch.cat([dh * z[:, F:] * da, dh * a], 1)
        return (dz @ s["w"].float()).to(t), (dz.T @ x).to(t)
    keep, scale = _keep(x.numel(), s["p"], s["seed"], s["offset"], x.device)
    y = torch.where(keep.view(x.shape), x * scale, torch.zeros_like(x))
    if s.get("residual"):
        y = y + s["r"].float()
    return (y.to(t),)


# ------------------------------------------------------------------ the package's calls

def _own(s):
    import convolution_backward_b200 as cb
    op = s["op"]
    if op == "ln_fwd":
        y = cb.layernorm_forward(s["x"], s["gamma"], s["beta"], eps=EPS, stats=s["stats"])
        return y if s["stats"] else (y,)
    if op == "ln_bwd":
        return cb.layernorm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"])
    if op == "gated_fwd":
        h = cb.gated_forward(s["x"], s["w"], act=s["act"], preact=s["keep"])
        return h if s["keep"] else (h,)
    if op == "gated_bwd":
        return cb.gated_backward(s["dh"], s["x"], s["z"], s["w"], act=s["act"])
    if op == "drop_fwd":
        return (cb.dropout_forward(s["x"], s["p"], s["seed"], s["offset"], residual=s.get("r")),)
    return (cb.dropout_backward(s["x"], s["p"], s["seed"], s["offset"]),)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    M, C, e, op = case["M"], case["C"], _BYTES[case["dtype"]], case["op"]
    n = M * C
    if op == "ln_fwd":
        return {"bytes": 2 * n * e + 2 * C * e + (8 * M if case["stats"] else 0), "flops": 8 * n}
    if op == "ln_bwd":
        return {"bytes": 3 * n * e + 3 * C * e + 8 * M, "flops": 14 * n}
    if op == "gated_fwd":
        F = case["F"]
        return {"bytes": e * (n + 2 * F * C + M * F * (3 if case["keep"] else 1)), "flops": 4 * M * F * C}
    if op == "gated_bwd":
        F = case["F"]
        return {"bytes": e * (2 * n + 4 * F * C + 3 * M * F), "flops": 8 * M * F * C}
    return {"bytes": n * e * (3 if case.get("residual") else 2), "flops": 2 * n}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_act(name, g):
    """act and act' in 64 bits, from forms other than the plain ones."""
    if name in ("silu", "sigmoid"):
        s = 0.5 + 0.5 * torch.tanh(0.5 * g)
        s = torch.where(g < -30, torch.exp(g), s)       # 1/(1+e^-g) = e^g(1 - e^g + ..)
        sp = 1 / (2 + torch.exp(g) + torch.exp(-g))     # the logistic density
        return (g * s, s + g * sp) if name == "silu" else (s, sp)
    if name == "relu":
        return torch.clamp(g, min=0), torch.where(g > 0, 1.0, 0.0).double()
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    v = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    dv = math.sqrt(2 / math.pi) * (1 + 0.134145 * g ** 2)
    s = 1 / (1 + torch.exp(-2 * v))                     # (1 + tanh v)/2
    return g * s, s + g * 2 * s * (1 - s) * dv


def _exact_keep(n, p, seed, offset):
    m32 = np.uint64(0xFFFFFFFF)
    sh = np.uint64(32)
    b = np.arange((n + 7) // 8, dtype=np.uint64)
    ctr = [b & m32, b >> sh, np.full_like(b, offset & 0xFFFFFFFF), np.full_like(b, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for r in range(10):
        k = [np.uint64((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF), np.uint64((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF)]
        a = ctr[0] * np.uint64(0xD2511F53)
        c = ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(c >> sh) ^ ctr[1] ^ k[0], c & m32, (a >> sh) ^ ctr[3] ^ k[1], a & m32]
    words = np.stack(ctr, 1).astype("<u4")
    draws = words.view("<u2").reshape(-1)[:n]
    thr = int(round(p * 65536))
    return draws >= thr, 65536.0 / (65536 - thr)


def exact(case, seed):
    s = prepare(case, seed)
    op, C = case["op"], case["C"]
    x = s["x"].double()
    if op == "ln_fwd":
        mean = x.mean(1)
        rstd = (x.var(1, unbiased=False) + EPS).rsqrt()
        n = (x - mean[:, None]) * rstd[:, None]
        y = torch.addcmul(s["beta"].double().expand_as(n), n, s["gamma"].double().expand_as(n))
        return (y, mean, rstd) if case["stats"] else (y,)
    if op == "ln_bwd":
        dy = s["dy"].double()
        r = s["rstd"].double()
        n = (x - s["mean"].double()[:, None]) * r[:, None]
        q = dy * s["gamma"].double()
        along = torch.einsum("mc,mc->m", q, n) / C
        dx = (q - q.mean(1)[:, None] - along[:, None] * n) * r[:, None]
        return dx, torch.einsum("mc,mc->c", dy, n), torch.einsum("mc->c", dy)
    if op == "gated_fwd":
        F = case["F"]
        w = s["w"].double()
        g, u = x @ w[:F].T, x @ w[F:].T
        h = _exact_act(case["act"], g)[0] * u
        return (h, torch.cat([g, u], 1)) if case["keep"] else (h,)
    if op == "gated_bwd":
        F = case["F"]
        w, z, dh = s["w"].double(), s["z"].double(), s["dh"].double()
        a, da = _exact_act(case["act"], z[:, :F])
        dg, du = dh * z[:, F:] * da, dh * a
        return dg @ w[:F] + du @ w[F:], torch.cat([dg.T @ x, du.T @ x], 0)
    keep, scale = _exact_keep(x.numel(), s["p"], s["seed"], s["offset"])
    y = x * scale * torch.from_numpy(keep).to(x.device).view(x.shape)
    if case.get("residual"):
        y = y + s["r"].double()
    return (y,)
