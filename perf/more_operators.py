"""What is measured of group norm, the AdamW step and the gradients' norm, with their plain forms.

A convolutional network's training program runs, between this package's convolution
gradients, group norm with an activation over the same NHWC rows; and behind them the norm
of all gradients and the optimizer's step over all parameters at once, with its states in
32 or in 8 bits.

``listed()`` names the cases, ``draw(rng)`` makes more of the same ranges, ``prepare`` makes
the inputs, ``run`` makes one pass (the plain form, or the package's calls when ``own`` is
set), ``work`` counts what the pass cannot do without and ``exact`` evaluates the
definition in 64 bits.

Definitions:
  group norm   x (N, S, C), G groups of D = C/G channels: mean, rstd = 1/sqrt(var + eps) over a
               group's S*D values of a sample, n = (x - mean)*rstd, z = n*gamma + beta,
               y = act(z); backward: dz = dy*act'(z), dgamma = sum dz*n, dbeta = sum dz over
               samples and positions, dx = rstd*(q - mean_g(q) - n*mean_g(q*n)) with q = dz*gamma.
  AdamW        g = scale*grad, m' = b1*m + (1 - b1)*g, v' = b2*v + (1 - b2)*g*g,
               p' = p*(1 - lr*wd) - lr*(m'/(1 - b1^t))/(sqrt(v'/(1 - b2^t)) + eps); p in fp32 (the
               master copy's where there is one), rounded to the parameter's type at the end.
  8-bit states Every 256 elements of a tensor share the fp32 maxima of |m| and v. With codes
               c in -127..127 and 0..255, m = (c*|c|*fl(1/127^2))*max|m| and
               v = (fl(c^4)*fl(1/255^4))*max v, each operation rounded to fp32. A step takes
               m', v' from fp32 operations in the order written in ``_moments``, and the codes
               from ``_code``: of the two neighbouring codes the nearer one's value (the lower at a
               tie), or the upper with probability (w - low)/(high - low). Its 16 bits are those
               of Philox-4x32-10 (J. Salmon et al., "Parallel random numbers: as easy as 1, 2, 3",
               2011) at counter (block, offset) and key seed: element i, counted with every tensor
               rounded up to 256 elements, takes word i % 4 of block i // 4, its low half for m and
               its high half for v. A v' above zero keeps a code above zero.
  norm         sqrt(sum of squares over all tensors), scale = min(1, max_norm/(norm + 1e-6)).
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
BLOCK = 256                     # elements that share a maximum
LR, B1, B2, AEPS, WD, STEP = 1e-3, 0.9, 0.999, 1e-8, 0.1, 1000
MAX_NORM = 1.0


def listed():
    return [
        # two images at the last 8x8 stage of an encoder: latency
        {"name": "gn_fwd_corner", "op": "gn_fwd", "dtype": "bf16", "N": 2, "S": 8 * 8, "C": 512, "G": 32, "act": "silu",
         "stats": False},
        # the 64x64 stage of a convolutional network, batch 16, training: 384 channels
        {"name": "gn_fwd_stage", "op": "gn_fwd", "dtype": "bf16", "N": 16, "S": 64 * 64, "C": 384, "G": 32, "act": "silu",
         "stats": True},
        # ragged rows of odd length in full precision, no activation
        {"name": "gn_fwd_odd", "op": "gn_fwd", "dtype": "f32", "N": 3, "S": 37 * 53, "C": 1001, "G": 7, "act": "none",
         "stats": True},
        # four images of the 16x16 stage, training
        {"name": "gn_bwd_corner", "op": "gn_bwd", "dtype": "bf16", "N": 4, "S": 16 * 16, "C": 768, "G": 32, "act": "silu"},
        # the early 112x112 stage, batch 32: many short rows, three channels a group
        {"name": "gn_bwd_early", "op": "gn_bwd", "dtype": "bf16", "N": 32, "S": 112 * 112, "C": 96, "G": 32, "act": "gelu"},
        # a ragged batch in half precision
        {"name": "gn_bwd_odd", "op": "gn_bwd", "dtype": "f16", "N": 5, "S": 37 * 53, "C": 328, "G": 8, "act": "gelu_tanh"},
        # one depthwise stage's parameters: latency
        {"name": "adamw_few", "op": "adamw", "dtype": "f32", "master": False, "tensors": 10, "elements": 100_000},
        # a network's parameters in mixed precision: some hundred tensors from biases to wide filters
        {"name": "adamw_net", "op": "adamw", "dtype": "bf16", "master": True, "tensors": 300, "elements": 60_000_000},
        # a smaller network, states in 8 bits, codes to the nearer value
        {"name": "adamw8_net", "op": "adamw8", "dtype": "f16", "master": True, "tensors": 160, "elements": 12_000_000,
         "rounding": "nearest"},
        # wide layers without a master copy, states in 8 bits, stochastic rounding
        {"name": "adamw8_wide", "op": "adamw8", "dtype": "bf16", "master": False, "tensors": 24, "elements": 80_000_000,
         "rounding": "stochastic"},
        # one depthwise stage's gradients: latency
        {"name": "norm_few", "op": "norm", "dtype": "f32", "tensors": 10, "elements": 100_000},
        # a network's gradients
        {"name": "norm_net", "op": "norm", "dtype": "bf16", "tensors": 300, "elements": 120_000_000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gn_fwd", "gn_fwd", "gn_bwd", "gn_bwd", "adamw", "adamw8", "norm"])
    case = {"op": op, "dtype": rng.choice(["f32", "bf16", "f16"])}
    if op.startswith("gn"):
        G, D = _log(rng, 1, 64), _log(rng, 1, 64)
        C = G * D
        N = _log(rng, 1, 32)
        most = 18_000_000 if op == "gn_fwd" else 25_000_000     # at four bytes no more than the largest listed
        # through a group of a few values goes only what cancellation leaves of a gradient
        least = -(-16 // D) if op == "gn_bwd" else 1
        S = _log(rng, least, max(least, min(65536, most // (N * C))))
        case.update(N=N, S=S, C=C, G=G, act=rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu", "sigmoid"]))
        if op == "gn_fwd":
            case["stats"] = rng.random() < 0.5
        return case
    case["tensors"] = _log(rng, 1, 400)
    most = {"adamw": 60_000_000, "adamw8": 40_000_000, "norm": 60_000_000}[op]
    case["elements"] = _log(rng, 400 * case["tensors"], most)
    if op != "norm":
        case["master"] = case["dtype"] != "f32" and rng.random() < 0.5
    if op == "adamw8":
        case["rounding"] = rng.choice(["nearest", "stochastic"])
    return case


def _sizes(case):
    """The tensors' element counts: spread over three decades, most of them whole rows, some odd."""
    rng = random.Random(case["tensors"] * 1_000_003 + case["elements"])
    share = [math.exp(rng.uniform(0, math.log(1000))) for _ in range(case["tensors"])]
    total = sum(share)
    got = []
    for s in share:
        n = max(1, int(s / total * case["elements"]))
        got.append(n if rng.random() < 0.3 or n < 64 else n // 64 * 64)
    return got


def _places(case):
    """(sizes, first elements) in one buffer where every tensor starts on a whole block, and its length."""
    sizes, first, at = _sizes(case), [], 0
    for n in sizes:
        first.append(at)
        at += -(-n // BLOCK) * BLOCK
    return sizes, first, at


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = _TYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device="cuda") * std + mean

    s = dict(case)
    if op.startswith("gn"):
        N, S, C, G = case["N"], case["S"], case["C"], case["G"]
        # activations: a common offset, channels of unlike scale, images of unlike brightness
        scale = normal(C, std=0.4).exp()
        s["x"] = (normal(N, S, C) * scale + normal(C, std=0.5) + normal(N, 1, 1, std=0.3)).to(t)
        s["gamma"] = normal(C, std=0.2, mean=1.0).to(t)
        s["beta"] = normal(C, std=0.2).to(t)
        if op == "gn_bwd":
            s["dy"] = normal(N, S, C, std=0.3).to(t)
            xg = s["x"].float().view(N, S, G, C // G)
            s["mean"] = xg.double().mean((1, 3)).float()
            d = xg - s["mean"][:, None, :, None]
            s["rstd"] = 1.0 / torch.sqrt((d * d).double().mean((1, 3)).float() + EPS)
        return s
    # a network's tensors, views of one buffer each kind, as a training program with flat buffers has them
    sizes, first, n = _places(case)
    length = torch.tensor(sizes, device="cuda")
    blocks = (length + BLOCK - 1) // BLOCK
    left = torch.repeat_interleave(length, blocks) - (
        torch.arange(n // BLOCK, device="cuda") - torch.repeat_interleave(blocks.cumsum(0) - blocks, blocks)) * BLOCK
    inside = torch.arange(BLOCK, device="cuda")[None, :] < left[:, None]            # not the padding
    unlike = torch.repeat_interleave(normal(len(sizes), std=0.7).exp(), blocks)[:, None]   # a scale of each tensor's own
    s["n"] = sum(sizes)

    def views(flat):
        return [flat[a:a + k] for a, k in zip(first, sizes)]

    def flat(v, dtype):
        return (v * inside).to(dtype).reshape(-1)

    s["g"] = flat(normal(n // BLOCK, BLOCK, std=2e-3) * unlike, t)
    s["grads"] = views(s["g"])
    if op == "norm":
        return s
    w = normal(n // BLOCK, BLOCK, std=0.05)
    s["p"] = flat(w, t)
    s["w"] = flat(w, torch.float32) if case["master"] else None
    s["scale"] = torch.full((), 0.25 + 0.5 * (seed % 7) / 7, device="cuda")        # the clipping factor
    m = normal(n // BLOCK, BLOCK, std=3e-4) * unlike
    v = (normal(n // BLOCK, BLOCK) * 1e-3 * unlike) ** 2 + (3e-4 * unlike) ** 2
    if op == "adamw":
        s["m"], s["v"] = flat(m, torch.float32), flat(v, torch.float32)
    else:
        m, v = m * inside, v * inside
        s["mmax"], s["vmax"] = m.abs().amax(1), v.amax(1)
        s["m"] = _code(m, s["mmax"], None, _square, 127.0).to(torch.int8).reshape(-1)
        s["v"] = _code(v, s["vmax"], None, _fourth, 255.0).to(torch.uint8).reshape(-1)
        s["m_out"], s["v_out"] = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        # random numbers are inputs: the generator's seed and offset
        s["seed"] = (0x9E3779B97F4A7C15 * (seed + 1) & (2 ** 64 - 1)) if case["rounding"] == "stochastic" else None
        s["offset"] = 5 + (seed << 33)
    if own:
        # the handle that a training program keeps: the lists of its parameters and states
        import convolution_backward_b200 as cb
        more = {"master": views(s["w"])} if case["master"] else {}
        if op == "adamw8":
            def maxima(flat):
                return [flat[a // BLOCK:-(-(a + k) // BLOCK)] for a, k in zip(first, sizes)]
            more["m_max"], more["v_max"] = maxima(s["mmax"]), maxima(s["vmax"])
            s["m_views"], s["v_views"] = views(s["m_out"]), views(s["v_out"])
        s["state"] = cb.AdamWState(views(s["p"]), views(s["m"]), views(s["v"]), **more)
    return s


# ------------------------------------------------------------------ plain forms

def _act(name, g):
    """act(g) and act'(g)."""
    if name == "none":
        return g, torch.ones_like(g)
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


def _square(c):
    return c * c


def _fourth(c):
    return (c * c) * (c * c)


def _stretch(top):
    """A power of two that brings the maxima to where their reciprocal is an ordinary number."""
    one = torch.ones_like(top)
    return torch.where(top < 2.0 ** -60, one * 2.0 ** 64, torch.where(top > 2.0 ** 60, one * 2.0 ** -64, one))


def _code(x, top, draws, value, most):
    """Codes (as fp32) of x (blocks, 256) whose magnitudes' maxima are top: value(c)/value(most)
    is what code c stands for. draws: 16 bits each, or None for the nearer code."""
    k = _stretch(top)
    inv = torch.where(top > 0, torch.reciprocal(top * k) * (value(torch.tensor(most)).item()), torch.zeros_like(top))
    w = (x.abs() * k[:, None]) * inv[:, None]
    low = torch.floor(torch.sqrt(w) if value is _square else torch.sqrt(torch.sqrt(w)))
    low = torch.where(value(low) > w, low - 1, low)
    low = torch.where(value(low + 1) <= w, low + 1, low)
    step = value(low + 1) - value(low)
    up = (w - value(low)) * 65536.0 > step * (32768.0 if draws is None else draws)
    c = torch.clamp(low + up.to(w.dtype), max=most)
    if value is _fourth:
        return torch.where((x > 0) & (c < 1), torch.ones_like(c), c)
    return torch.where(x < 0, -c, c)


def _moments(s):
    """The values that 8-bit states stand for, (blocks, 256)."""
    c = s["m"].float().view(-1, BLOCK)
    m = ((c * c.abs()) * (1 / 16129)) * s["mmax"][:, None]
    v = (_fourth(s["v"].float().view(-1, BLOCK)) * (1 / 4228250625)) * s["vmax"][:, None]
    return m, v


def _mulhilo(a, const):
    """High and low 32 bits of a * const for 32-bit values held in int64."""
    lo_p = (a & 0xFFFF) * const
    hi_p = (a >> 16) * const
    mid = hi_p + (lo_p >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (lo_p & 0xFFFF)


def _draws(n, seed, offset, device):
    """Two 16-bit draws for each of n elements (a multiple of 256), as fp32 (blocks, 256)."""
    b = torch.arange(n // 4, device=device, dtype=torch.int64)
    c0, c1 = b & 0xFFFFFFFF, b >> 32
    c2 = torch.full_like(b, offset & 0xFFFFFFFF)
    c3 = torch.full_like(b, offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    word = torch.stack([c0, c1, c2, c3], 1).reshape(-1, BLOCK)
    return (word & 0xFFFF).float(), (word >> 16).float()


def _plain(s):
    op = s["op"]
    if op == "gn_fwd" or op == "gn_bwd":
        N, S, C, G = s["N"], s["S"], s["C"], s["G"]
        t = s["x"].dtype
        x = s["x"].float().view(N, S, G, C // G)
        gamma, beta = s["gamma"].float().view(G, C // G), s["beta"].float().view(G, C // G)
        count = S * (C // G)
        if op == "gn_fwd":
            mean = x.sum((1, 3), keepdim=True) / count
            d = x - mean
            rstd = 1.0 / torch.sqrt((d * d).sum((1, 3), keepdim=True) / count + EPS)
            y = _act(s["act"], d * rstd * gamma + beta)[0].to(t).view(N, S, C)
            return (y, mean.view(N, G), rstd.view(N, G)) if s["stats"] else (y,)
        rstd = s["rstd"][:, None, :, None]
        n = (x - s["mean"][:, None, :, None]) * rstd
        dz = s["dy"].float().view(N, S, G, C // G) * _act(s["act"], n * gamma + beta)[1]
        q = dz * gamma
        dx = rstd * (q - q.sum((1, 3), keepdim=True) / count - n * ((q * n).sum((1, 3), keepdim=True) / count))
        return dx.to(t).view(N, S, C), (dz * n).sum((0, 1)).to(t).view(C), dz.sum((0, 1)).to(t).view(C)
    if op == "norm":
        norm = torch.sqrt((s["g"].double() ** 2).sum()).float()
        return norm, torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)
    g = s["g"].float() * s["scale"]
    w = s["w"] if s["w"] is not None else s["p"].float()
    if op == "adamw":
        m, v = s["m"], s["v"]
    else:
        g, w = g.view(-1, BLOCK), w.view(-1, BLOCK)
        m, v = _moments(s)
    m = m * B1 + g * (1 - B1)
    v = v * B2 + (g * (1 - B2)) * g
    step = (m / (1 - B1 ** STEP)) / (torch.sqrt(v / (1 - B2 ** STEP)) + AEPS)
    w = (w * (1 - LR * WD) - step * LR).view(-1)
    if s["w"] is not None:
        s["w"].copy_(w)
    s["p"].copy_(w)
    if op == "adamw":
        s["m"].copy_(m)
        s["v"].copy_(v)
        return (s["p"], s["m"], s["v"]) if s["w"] is None else (s["p"], s["m"], s["v"], s["w"])
    dm = dv = None
    if s["seed"] is not None:
        dm, dv = _draws(g.numel(), s["seed"], s["offset"], g.device)
    s["mmax"].copy_(m.abs().amax(1))
    s["vmax"].copy_(v.amax(1))
    s["m"].copy_(_code(m, s["mmax"], dm, _square, 127.0).view(-1))
    s["v"].copy_(_code(v, s["vmax"], dv, _fourth, 255.0).view(-1))
    m, v = _moments(s)      # what the 8-bit states stand for now
    s["m_out"].copy_(m.view(-1))
    s["v_out"].copy_(v.view(-1))
    return (s["p"], s["m_out"], s["v_out"]) if s["w"] is None else (s["p"], s["m_out"], s["v_out"], s["w"])


# ------------------------------------------------------------------ the package's calls

def _own(s):
    import convolution_backward_b200 as cb
    op = s["op"]
    act = None if s.get("act") == "none" else s.get("act")
    if op == "gn_fwd":
        y = cb.groupnorm_forward(s["x"], s["G"], s["gamma"], s["beta"], eps=EPS, act=act, stats=s["stats"])
        return y if s["stats"] else (y,)
    if op == "gn_bwd":
        return cb.groupnorm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"], s["beta"], act=act)
    if op == "norm":
        return cb.grad_norm(s["grads"], MAX_NORM)
    if op == "adamw":
        cb.adamw_step(s["state"], s["grads"], STEP, LR, (B1, B2), AEPS, WD, grad_scale=s["scale"])
        return (s["p"], s["m"], s["v"]) if s["w"] is None else (s["p"], s["m"], s["v"], s["w"])
    cb.adamw_step(s["state"], s["grads"], STEP, LR, (B1, B2), AEPS, WD, grad_scale=s["scale"], seed=s["seed"],
                  offset=s["offset"])
    cb.adamw_moments(s["state"], out=(s["m_views"], s["v_views"]))     # what the 8-bit states stand for now
    return (s["p"], s["m_out"], s["v_out"]) if s["w"] is None else (s["p"], s["m_out"], s["v_out"], s["w"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    e, op = _BYTES[case["dtype"]], case["op"]
    if op.startswith("gn"):
        n, C = case["N"] * case["S"] * case["C"], case["C"]
        stats = 8 * case["N"] * case["G"]
        if op == "gn_fwd":
            return {"bytes": 2 * n * e + 2 * C * e + (stats if case["stats"] else 0), "flops": 12 * n}
        return {"bytes": 3 * n * e + 4 * C * e + stats, "flops": 30 * n}
    n = sum(_sizes(case))
    if op == "norm":
        return {"bytes": n * e, "flops": 2 * n}
    weights = e + (2 * 4 + e if case["master"] else 2 * e)     # the gradient; master read and written, p written
    if op == "adamw":
        return {"bytes": n * (weights + 16), "flops": 16 * n}
    # codes read and written, the maxima, and the moments they stand for written out
    return {"bytes": n * (weights + 4 + 8) + 16 * (n // BLOCK), "flops": 60 * n}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_act(name, g):
    """act and act' in 64 bits, from forms other than the plain ones."""
    if name == "none":
        return g, torch.ones((), dtype=g.dtype, device=g.device)
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


def _exact_draws(n, seed, offset):
    """The generator's 32-bit words for n elements, in numpy's unsigned arithmetic."""
    m32, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    b = np.arange(n // 4, dtype=np.uint64)
    ctr = [b & m32, b >> sh, np.full_like(b, offset & 0xFFFFFFFF), np.full_like(b, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for r in range(10):
        k = [np.uint64((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF), np.uint64((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF)]
        a = ctr[0] * np.uint64(0xD2511F53)
        c = ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(c >> sh) ^ ctr[1] ^ k[0], c & m32, (a >> sh) ^ ctr[3] ^ k[1], a & m32]
    return torch.from_numpy(np.stack(ctr, 1).reshape(-1).astype(np.int64))


def _r(x):
    """A result in 64 bits rounded to fp32, where the definition says so (sums, products, quotients and roots of fp32
    values that are formed in 64 bits and then rounded are the ones that fp32 operations give)."""
    return x.float().double()


def _exact_table(power, most, device):
    return _r(_r(torch.arange(most + 2, device=device).double() ** 2) ** (power // 2))


def _exact_quantised(x, power, most, draw):
    """What x >= 0 (blocks, 256) stands for once held as (c/most)^power of its block's largest value: the codes by
    search in their table, their values in 64 bits."""
    table = _exact_table(power, most, x.device)
    top = x.amax(1, keepdim=True)
    k = torch.where(top < 2.0 ** -60, 2.0 ** 64, torch.where(top > 2.0 ** 60, 2.0 ** -64, 1.0)).double()
    inv = torch.where(top > 0, _r(_r(1 / (top * k)) * table[most]), torch.zeros_like(top))
    w = _r(_r(x * k) * inv)
    low = torch.searchsorted(table, w, right=True) - 1
    step = _r(table[(low + 1).clamp(max=most + 1)] - table[low])
    low = low + (_r(w - table[low]) * 65536 > _r(step * (32768 if draw is None else draw)))
    low = low.clamp(max=most)
    if power == 4:
        low = torch.where((x > 0) & (low < 1), torch.ones_like(low), low)
    return (low.double() / most) ** power * top


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("gn"):
        N, S, C, G = case["N"], case["S"], case["C"], case["G"]
        D = C // G
        x = s["x"].double()
        gamma, beta = s["gamma"].double(), s["beta"].double()
        if op == "gn_fwd":
            by = x.view(N, S, G, D).transpose(1, 2).reshape(N, G, S * D)
            mean = by.mean(2)
            rstd = (by.var(2, unbiased=False) + EPS).rsqrt()
            del by
            a = rstd.repeat_interleave(D, 1) * gamma                # y = act(a x + b)
            b = beta - mean.repeat_interleave(D, 1) * a
            y = _exact_act(case["act"], torch.addcmul(b[:, None, :], x, a[:, None, :]))[0]
            return (y, mean, rstd) if case["stats"] else (y,)
        mean = s["mean"].double().repeat_interleave(D, 1)[:, None, :]
        rstd = s["rstd"].double().repeat_interleave(D, 1)[:, None, :]
        n = (x - mean) * rstd
        dz = s["dy"].double() * _exact_act(case["act"], torch.addcmul(beta, n, gamma))[1]
        by_sample, along = dz.sum(1), torch.einsum("nsc,nsc->nc", dz, n)
        m1 = (by_sample * gamma).view(N, G, D).sum(2).repeat_interleave(D, 1)[:, None, :] / (S * D)
        m2 = (along * gamma).view(N, G, D).sum(2).repeat_interleave(D, 1)[:, None, :] / (S * D)
        return (dz * gamma - m1 - n * m2) * rstd, along.sum(0), by_sample.sum(0)
    g = s["g"].double()
    if op == "norm":
        norm = torch.linalg.vector_norm(g)
        return norm, torch.where(norm + 1e-6 > MAX_NORM, MAX_NORM / (norm + 1e-6), torch.ones_like(norm))
    g = g * s["scale"].double()
    w = (s["w"] if case["master"] else s["p"]).double()
    if op == "adamw":
        m, v = s["m"].double(), s["v"].double()
        m = torch.lerp(g, m, B1)
        v = torch.lerp(g * g, v, B2)
    else:       # fp32 moments, in the definition's operations
        f32 = lambda c: torch.tensor(c, device=g.device).double()
        c, d = s["m"].double(), s["v"].double()
        g = _r(g)
        m = _r(_r(c * c.abs() * f32(1 / 16129)) * s["mmax"].double().repeat_interleave(BLOCK))
        v = _exact_table(4, 255, g.device)[d.long()]
        v = _r(_r(v * f32(1 / 4228250625)) * s["vmax"].double().repeat_interleave(BLOCK))
        m = _r(_r(m * f32(B1)) + _r(g * f32(1 - B1)))
        v = _r(_r(v * f32(B2)) + _r(_r(g * f32(1 - B2)) * g))
    w = w - LR * (WD * w + m / -math.expm1(STEP * math.log(B1)) / ((v / -math.expm1(STEP * math.log(B2))).sqrt() + AEPS))
    if op == "adamw8":
        dm = dv = None
        if s["seed"] is not None:
            words = _exact_draws(g.numel(), s["seed"], s["offset"]).to(g.device).view(-1, BLOCK)
            dm, dv = (words & 0xFFFF).double(), (words >> 16).double()
        m, v = m.view(-1, BLOCK), v.view(-1, BLOCK)
        m = (_exact_quantised(m.abs(), 2, 127, dm) * torch.sign(m)).view(-1)
        v = _exact_quantised(v, 4, 255, dv).view(-1)
    return (w, m, v) if not case["master"] else (w, m, v, w)
