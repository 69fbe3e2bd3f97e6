"""The residual branch's operators where they can go wrong: activations far out, the ends of the
types' ranges, infinities, layer norm's and the gated gradients' loops over many rows and tiles.
Against the definitions in 64 bits.

Tolerances, elementwise (u, eta: the type's half step relative to the value and half its
smallest subnormal; e = 2^-24), beyond those of test_branch_ops.py and test_gated.py:
  act, act'   The exponential's argument t carries up to three roundings, so the exponential
              is off relatively by 3 t e, and the approximate exponential, reciprocal and
              products by less than 20 e more: rel = (20 + 4 t) e with t = |g| (silu,
              sigmoid), g^2/2 (gelu; its fitted tail adds 2.5e-7 = 4.2 e), 2|v| (the tanh
              form).  1 - s is off by 2 e absolutely where s < 1, which is for t < 18 only:
              silu' by 2 e t s, the tanh form's by 2 e (2|g| dv/dg) s.  What lies below
              2^-126 may be zero, and is multiplied by at most 90.
  dZ          three products more.  On the tensor cores it is rounded once more: u |dz| and,
              f16, half a subnormal step: 2^-25, or where dZ is scaled 2^-39 of its largest value.
"""
import os
import subprocess
import sys

import numpy as np
import pytest

import convolution_backward_b200 as cb
import test_branch_ops as tb
import test_gated as tg
from oracle import branch

torch = pytest.importorskip("torch")

E32 = 2.0 ** -24
TYPES = tb.TYPES
HALF = tg.TYPES
TINY = 90 * 2.0 ** -126


def act64(name, g):
    """(act, act', rel, abs of act'): the activation in 64 bits and its fp32 evaluation's errors."""
    if name == "relu":
        return np.maximum(g, 0.0), (g > 0).astype(np.float64), 0 * g, 0 * g

    def logistic(v):     # s(v), s(v) s(-v)
        x = np.exp(-np.abs(v))
        return np.where(v >= 0, 1.0, x) / (1 + x), x / (1 + x) ** 2

    if name in ("silu", "sigmoid"):
        t = np.abs(g)
        s, p = logistic(g)
        a, d, mag = (g * s, s + g * p, s + t * p) if name == "silu" else (s, p, p)
        near = np.where(t < 18, 2 * E32 * t * s, 0.0) if name == "silu" else 0 * g
    elif name == "gelu":
        t = g * g / 2
        cdf = 0.5 * torch.special.erfc(torch.from_numpy(-g / np.sqrt(2.0))).numpy()
        phi = np.exp(-t) / np.sqrt(2 * np.pi)
        a, d, mag, near = g * cdf, cdf + g * phi, cdf + np.abs(g) * phi, 0 * g
    else:
        k = np.sqrt(2 / np.pi)
        v, dv = k * (g + 0.044715 * g ** 3), k * (1 + 3 * 0.044715 * g * g)
        t = 2 * np.abs(v)
        s, p = logistic(2 * v)
        a, d, mag = g * s, s + 2 * g * p * dv, s + 2 * np.abs(g) * p * dv
        near = np.where(t < 18, 4 * E32 * np.abs(g) * dv * s, 0.0)
    rel = (25 + 4 * t) * E32
    return a, d, rel, np.where(mag > 0, rel * mag, 0.0) + near


def dz64(act, dh, z):
    """(dZ, the fp32 evaluation's error)."""
    F = dh.shape[1]
    g, u = z[:, :F], z[:, F:]
    a, d, rel, ed = act64(act, g)
    dz = np.concatenate([dh * u * d, dh * a], axis=1)
    with np.errstate(invalid="ignore"):
        ea = np.where(a != 0, rel * np.abs(a), 0.0)
    err = np.concatenate([np.abs(dh * u) * (ed + TINY), np.abs(dh) * (ea + TINY)], axis=1) + 4 * E32 * np.abs(dz)
    return dz, err


def tails(dtype):
    """Gates from zero to the type's largest value, both signs: 64 of them."""
    top = float(torch.finfo(HALF[dtype][0]).max)
    g = [2.0 ** -20, 0.01, 0.1, 0.5, 0.75, 1.0, 1.28, 1.5, 2, 2.5, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 14, 16, 17, 20, 24, 30, 60,
         80, 300, 1e4, 6e4]
    return np.array([0.0, *g, *[-v for v in g], top if top > 1e5 else 5e4])


# ----------------------------------------------------------- activations far out

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(HALF))
@pytest.mark.parametrize("act", tg.ACTS)
def test_activations_to_the_ends(act, dtype):
    """X is the identity, so that the pre-activations are W's own values: H = act(g) u."""
    t, u, eta = HALF[dtype]
    g = torch.from_numpy(tails(dtype)).to(t)
    other = torch.tensor([1.0, -0.5, 0.375, 1.0])
    F = 72
    w = torch.cat([g.expand(F, 64), other.repeat(18)[:, None].expand(F, 64).to(t)]).contiguous().cuda()
    x = torch.eye(64, dtype=t, device="cuda")
    for M in (64, 30, 7, 1):    # the pair kernel, the kernels of few rows
        for lo in range(0, 64 if M > 1 else 0, M) or (0, 20, 50):
            rows = x[lo:lo + M]
            h, z = cb.gated_forward(rows, w, act=act, preact=True)
            Z = w.t()[lo:lo + M]
            assert torch.equal(z, Z)
            Z = tg.to64(Z)
            a, _, rel, _ = act64(act, Z[:, :F])
            ref = a * Z[:, F:]
            tg.within(h, ref, u * np.abs(ref) + 1.01 * (rel + 2 * E32) * np.abs(ref) + TINY + eta, f"M={M} from {lo}")
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("F", [64, 72])      # dZ in fp32; rounded for the tensor cores
@pytest.mark.parametrize("dtype", list(HALF))
@pytest.mark.parametrize("act", tg.ACTS)
def test_derivatives_to_the_ends(act, dtype, F):
    """X and the gate's rows of W are identities: dW is dZ^T, dX the gate's part of dZ."""
    t, u, eta = HALF[dtype]
    mk = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()
    r = np.random.default_rng(7)
    g = np.broadcast_to(tails(dtype)[:, None], (64, F))
    other = np.broadcast_to(np.resize([1.0, -0.5, 768.0, 0.0], F), (64, F))
    dh = mk(np.resize([1.0, -0.75, 0.5], (64, F)) * r.choice([-1.0, 1.0], size=(64, F)))
    z = mk(np.concatenate([g, other], axis=1))
    x = torch.eye(64, dtype=t, device="cuda")
    w = torch.zeros(2 * F, 64, dtype=t, device="cuda")
    w[:64] = x
    dx, dw = cb.gated_backward(dh, x, z, w, act=act)
    cb.check_status()
    dz, err = dz64(act, tg.to64(dh), tg.to64(z))
    bound = 2 * u * (1 + u) * np.abs(dz) + 1.01 * err + 2 * eta
    tg.within(dw.t(), dz, bound, "dw")
    tg.within(dx, dz[:, :64], bound[:, :64], "dx")


# ------------------------------------------- the gated gradients' range and loops

def _gpu64(*ts):
    return [t.detach().double() for t in ts]


def _within(got, ref, bound, what):
    """As test_gated.within, on the GPU."""
    bad = ~((got.double() - ref).abs() <= bound)
    if bool(bad.any()):
        i = int(torch.argmax(torch.where(bad, (got.double() - ref).abs() / bound, torch.zeros_like(ref)).flatten()))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, worst at {i}: got {got.flatten()[i].item()!r}, "
                             f"want {ref.flatten()[i].item()!r}, bound {bound.flatten()[i].item()!r}")


def _check_gated_backward(dh, x, z, w, dtype, dx, dw, what):
    """silu, on the GPU in 64 bits."""
    _, u, eta = HALF[dtype]
    DH, X, Z, W = _gpu64(dh, x, z, w)
    F = DH.shape[1]
    g, uu = Z[:, :F], Z[:, F:]
    t = g.abs()
    s, p = torch.sigmoid(g), torch.sigmoid(g) * torch.sigmoid(-g)
    rel = (25 + 4 * t) * E32
    dz = torch.cat([DH * uu * (s + g * p), DH * g * s], 1)
    e = torch.cat([(DH * uu).abs() * (rel * (s + t * p) + 2 * E32 * t.clamp(max=18) * s), DH.abs() * t * s * rel], 1)
    top = float(dz.abs().max())
    least = 0.0 if dtype != "f16" else 2.0 ** -25 if 2.0 ** -10 <= top <= 65504 else top * 2.0 ** -39
    e = u * dz.abs() + 1.01 * (e + 4 * E32 * dz.abs()) + least
    for got, ref, err, terms in ((dx, dz @ W, e @ W.abs(), 2 * F * (dz.abs() @ W.abs())),
                                 (dw, dz.t() @ X, e.t() @ X.abs(), X.shape[0] * (dz.abs().t() @ X.abs()))):
        if got is None:
            continue
        _within(got, ref, u * ref.abs() + (1 + u) * (err + 1.01 * E32 * terms) + eta, f"{what} {tuple(ref.shape)}")
        # two roundings of at most u, evenly spread: in norm sqrt(2/3) u, a tenth for the rest
        assert float((got.double() - ref).norm() / ref.norm()) <= 1.1 * (2 / 3) ** 0.5 * u, what


# (few values), (pairs' tiles for dX, whole sums for dW), (dX's sums split), (dW's rows split)
RANGE_SHAPES = [(16, 72, 40), (300, 136, 264), (300, 1096, 1208), (2600, 264, 72)]


def _scaled(shape, dtype, seed, ks):
    """x, w, dh, z with dH, U, X and W scaled by powers of two."""
    x, w, dh = tg._inputs(*shape, dtype, seed)
    z = cb.gated_forward(x, w, preact=True)[1]
    a, b, c, d = (2.0 ** k for k in ks)
    F = shape[2]
    z = z.clone()
    z[:, F:] *= b
    return x * c, w * d, dh * a, z


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(HALF))
@pytest.mark.parametrize("ks", [(9, 8, -12, -12), (-14, -6, 8, 8), (-8, -4, 4, 4)], ids=["large", "small", "middling"])
@pytest.mark.parametrize("shape", RANGE_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gated_backward_over_the_range(shape, ks, dtype):
    """dZ above f16's largest value and among its subnormals, between results that are neither."""
    x, w, dh, z = _scaled(shape, dtype, 5, ks)
    dx, dw = cb.gated_backward(dh, x, z, w)
    cb.check_status()
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    _check_gated_backward(dh, x, z, w, dtype, dx, dw, str(ks))
    for only in (dict(weight_grad=False), dict(input_grad=False)):
        got = cb.gated_backward(dh, x, z, w, **only)
        assert all(p is None or torch.equal(p, q) for p, q in zip(got, (dx, dw)))


@pytest.mark.gpu
def test_gated_backward_range_in_a_graph():
    """One captured backward pass replayed with gradients of unlike size."""
    cases = [_scaled((300, 136, 264), "f16", 5, ks) for ks in ((9, 8, -12, -12), (0, 0, 0, 0), (-14, -6, 8, 8))]
    want = [[t.clone() for t in cb.gated_backward(dh, x, z, w)] for x, w, dh, z in cases]
    x, w, dh, z = (t.clone() for t in cases[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = cb.gated_backward(dh, x, z, w)
    for i in (0, 1, 2, 1, 0):
        for into, of in zip((x, w, dh, z), cases[i]):
            into.copy_(of)
        g.replay()
        assert all(torch.equal(p, q) for p, q in zip(out, want[i]))
    cb.check_status()


# More units than the GPU has SM pairs: dX's tiles, dW's tiles, dW's narrow tiles
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(HALF))
@pytest.mark.parametrize("shape", [(2600, 2056, 264), (12000, 264, 72), (300, 2056, 1160), (700, 3000, 1096), (130, 104, 9704),
                                   (20000, 72, 24)], ids=lambda s: "x".join(map(str, s)))
def test_gated_backward_more_tiles_than_pairs(shape, dtype):
    x, w, dh = tg._inputs(*shape, dtype, seed=3)
    z = cb.gated_forward(x, w, preact=True)[1]
    dx, dw = cb.gated_backward(dh, x, z, w)
    cb.check_status()
    _check_gated_backward(dh, x, z, w, dtype, dx, dw, str(shape))
    again = cb.gated_backward(dh, x, z, w)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(HALF))
@pytest.mark.parametrize("shape", [(16, 72, 40), (300, 136, 264)], ids=lambda s: "x".join(map(str, s)))
def test_gated_backward_infinities(shape, dtype):
    """A NaN or an infinity spoils its own row of dX and its own column's rows of dW."""
    M, C, F = shape
    x, w, dh = tg._inputs(*shape, dtype, seed=3)
    z = cb.gated_forward(x, w, preact=True)[1]
    dh[5, 9] = 0
    clean = cb.gated_backward(dh, x, z, w)
    rows = [m for m in range(M) if m != 5]
    outs = [j for j in range(2 * F) if j % F != 9]
    for bad in (float("nan"), float("inf")):
        d = dh.clone()
        d[5, 9] = bad
        dx, dw = cb.gated_backward(d, x, z, w)
        assert torch.equal(dx[rows], clean[0][rows]) and torch.equal(dw[outs], clean[1][outs])
        assert not torch.isfinite(dx[5]).any() and not torch.isfinite(dw[[9, F + 9]]).any()
    for act in tg.ACTS:     # an overflowed pre-activation
        d = dh.clone()
        d[5, 9] = 1
        zz = z.clone()
        zz[5, 9] = float("-inf")
        clean = cb.gated_backward(dh, x, z, w, act=act)
        dx, dw = cb.gated_backward(d, x, zz, w, act=act)
        assert torch.equal(dx[rows], clean[0][rows]) and torch.equal(dw[outs], clean[1][outs])
        if act in ("relu", "sigmoid"):
            assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
        else:
            assert torch.isnan(dx[5]).all() and torch.isnan(dw[[9, F + 9]]).all()
    cb.check_status()


# ------------------------------------------------------------------------ layer norm

def _ln_fwd_check(x, g, b, eps, dtype, y, mean, rstd, what):
    """test_branch_ops._check_fwd on the GPU."""
    _, u, eta = TYPES[dtype]
    X, G, B = _gpu64(x, g, b)
    C = X.shape[1]
    K = tb.chain(C)
    rm = X.mean(1)
    rr = 1 / torch.sqrt(((X - rm[:, None]) ** 2).mean(1) + eps)
    em = (K + 1) * E32 * X.abs().mean(1) + E32 * rm.abs()
    er = ((K / 2 + 4) * E32 + 0.5 * (em * rr) ** 2) * rr
    _within(mean, rm, em, what + " mean")
    _within(rstd, rr, er, what + " rstd")
    n = (X - rm[:, None]) * rr[:, None]
    ey = ((em * rr)[:, None] + n.abs() * ((K / 2 + 8) * E32 + 0.5 * (em * rr)[:, None] ** 2)) * G.abs() \
        + 2 * E32 * ((n * G).abs() + B.abs())
    ry = n * G + B
    _within(y, ry, u * ry.abs() + (1 + u) * 1.01 * ey + eta, what + " y")


def _ln_bwd_check(dy, x, g, mean, rstd, dtype, got, what):
    """test_branch_ops._check_bwd on the GPU."""
    M, C = x.shape
    _, u, eta = TYPES[dtype]
    DY, X, G, m, r = _gpu64(dy, x, g, mean, rstd)
    n, q = (X - m[:, None]) * r[:, None], DY * G
    mq, mqn = q.mean(1, keepdim=True), (q * n).mean(1, keepdim=True)
    K = tb.chain(C)
    ref = r[:, None] * (q - mq - n * mqn)
    ex = r[:, None] * E32 * (5 * q.abs() + (K + 6) * q.abs().mean(1, keepdim=True)
                             + n.abs() * (K + 12) * (q * n).abs().mean(1, keepdim=True))
    _within(got[0], ref, u * ref.abs() + (1 + u) * 1.01 * ex + eta, what + " dx")
    k = (M + 64) * E32 * 1.01
    for o, terms, more, name in ((got[1], DY * n, 3 * E32, "dgamma"), (got[2], DY, 0.0, "dbeta")):
        if o is None:
            continue
        ref = terms.sum(0)
        _within(o, ref, u * ref.abs() + (1 + u) * (k + more) * terms.abs().sum(0) + eta, f"{what} {name}")


def _ln_rows(M, C, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    t = TYPES[dtype][0]
    x = (rnd(M, C) * (0.4 * rnd(C)).exp() + 0.5 * rnd(C)).to(t)
    return x, (1 + 0.2 * rnd(C)).to(t), (0.2 * rnd(C)).to(t), rnd(M, C).to(t)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])      # f16 holds no such rows
@pytest.mark.parametrize("k", [-66, 60], ids=["tiny", "huge"])
@pytest.mark.parametrize("shape", [(9, 96), (40, 1001), (5, 768), (3, 20001)], ids=lambda s: "x".join(map(str, s)))
def test_layernorm_backward_far_statistics(shape, k, dtype):
    """Rows of 2^-66 and of 2^60: the gradient scales with 1/spread, whose square fp32 does not hold."""
    x, g, b, dy = _ln_rows(*shape, dtype, seed=4)
    x = (x.float() * 2.0 ** k).to(x.dtype)
    X = x.double()
    mean = X.mean(1).float()
    rstd = (1 / (X.var(1, unbiased=False)).sqrt()).float()
    got = cb.layernorm_backward(dy, x, mean, rstd, g)
    cb.check_status()
    _ln_bwd_check(dy, x, g, mean, rstd, dtype, got, f"2^{k}")


# Enough rows that every block takes several steps of them, the last one a part: within a warp and across warps, on
# and off the 16-byte grid, rows shorter than a vector, vectors per thread from one to the most.
MANY = [(40_009, 1), (40_009, 3), (40_009, 7), (40_009, 9), (30_011, 13), (30_011, 33), (30_011, 57), (30_011, 100),
        (20_011, 201), (20_011, 385), (240_007, 8), (240_007, 16), (160_009, 64), (80_021, 96), (20_021, 384), (20_021, 640),
        (9_001, 771), (9_001, 1536), (5_003, 2048), (3_001, 4104), (3_001, 4099), (1_801, 8200)]


def _many(shape, dtype, edge):
    M, C = shape
    x, g, b, dy = _ln_rows(M, C, dtype, seed=M + C)
    if C == 1:
        b = b + 1
    y, mean, rstd = cb.layernorm_forward(x, g, b, eps=1e-5, stats=True)
    grads = cb.layernorm_backward(dy, x, mean, rstd, g)
    cb.check_status()
    _ln_fwd_check(x, g, b, 1e-5, dtype, y, mean, rstd, edge)
    _ln_bwd_check(dy, x, g, mean, rstd, dtype, grads, edge)
    return x, g, b, dy, (y, mean, rstd), grads


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", MANY, ids=lambda s: "x".join(map(str, s)))
def test_layernorm_many_rows(shape, dtype):
    x, g, b, dy, want, grads = _many(shape, dtype, "many rows")
    z = x.clone()               # rows in flight are not disturbed by results written over their tensor
    got = cb.layernorm_forward(z, g, b, eps=1e-5, stats=True, out=z)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    for which in (0, 1):
        d, z = dy.clone(), x.clone()
        got = cb.layernorm_backward(d, z, want[1], want[2], g, out=d if which == 0 else z)
        assert all(torch.equal(p, q) for p, q in zip(got, grads))
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(40_009, 3), (40_009, 9), (30_011, 57), (20_011, 201), (240_007, 8), (80_021, 96), (20_021, 640),
                                   (9_001, 1536), (3_001, 4099)], ids=lambda s: "x".join(map(str, s)))
def test_layernorm_many_rows_every_store_in_bounds(shape, dtype, monkeypatch):
    path = os.path.join(os.path.dirname(cb.library_path()), "libdgrad_debug.so")
    if not os.path.exists(path):
        pytest.skip("libdgrad_debug.so not built")
    monkeypatch.setattr(cb, "_LIB_PATH", path)
    monkeypatch.setattr(cb, "_lib", None)
    _many(shape, dtype, "debug")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 8, 9, 33, 64, 96, 100, 201, 384, 768, 1001, 2048])
def test_layernorm_many_rows_take_every_sm(C, dtype):
    """The workspace holds 8 C bytes per block: 20000 rows are a block's work for every SM."""
    for i in range(200):
        M = int(20000 * 1.02 ** i)
        assert cb.layernorm_backward_workspace_bytes(M, C, dtype) // (8 * C) >= 140, M


@pytest.mark.parametrize("case", [(torch.bfloat16, 9, 4736), (torch.bfloat16, 33, 4736), (torch.bfloat16, 100, 4736),
                                  (torch.bfloat16, 64, 9472), (torch.bfloat16, 96, 18944), (torch.float32, 9, 4736),
                                  (torch.float32, 100, 2368), (torch.float32, 64, 9472)], ids=lambda c: f"{c[0]}x{c[1]}")
def test_layernorm_blocks_where_rows_pass_one_step(case):
    """One row more than a step for every resident block: about as many blocks, not a few with many steps."""
    dtype, C, M = case
    blocks = lambda m: cb.layernorm_backward_workspace_bytes(m, C, dtype) // (8 * C)
    for m in range(M, M + 3 * M // 2, 37):
        assert 2 * blocks(m + 1) >= blocks(m), m


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(9, 96), (40, 201), (60, 1001), (5000, 96), (5, 20001)], ids=lambda s: "x".join(map(str, s)))
def test_layernorm_backward_infinities(shape, dtype):
    """A NaN or an infinity in dY spoils its own row of dX and its own columns of dgamma and dbeta."""
    M, C = shape
    x, g, b, dy = _ln_rows(M, C, dtype, seed=4)
    _, mean, rstd = cb.layernorm_forward(x, g, b, stats=True)
    dy[3, 11] = 0
    clean = cb.layernorm_backward(dy, x, mean, rstd, g)
    rows, cols = [m for m in range(M) if m != 3], [c for c in range(C) if c != 11]
    for bad in (float("nan"), float("inf"), float("-inf")):
        d = dy.clone()
        d[3, 11] = bad
        dx, dg, db = cb.layernorm_backward(d, x, mean, rstd, g)
        assert torch.equal(dx[rows], clean[0][rows])
        assert torch.equal(dg[cols], clean[1][cols]) and torch.equal(db[cols], clean[2][cols])
        assert not torch.isfinite(dx[3]).any() and not torch.isfinite(dg[11]) and not torch.isfinite(db[11])
    cb.check_status()


# ------------------------------------------------------------------------- dropout

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n", [64, 100_003])
def test_dropout_keeps_the_sign_of_zero(n, dtype):
    x = torch.full((n,), -0.0, dtype=TYPES[dtype][0], device="cuda")
    assert torch.signbit(cb.dropout_forward(x, 0.0, 3)).all()
    keep = torch.from_numpy(branch.dropout_keep(n, 0.4, 3, 0)[0]).cuda()
    assert torch.equal(torch.signbit(cb.dropout_backward(x, 0.4, 3)), keep)
    assert torch.signbit(cb.dropout_forward(x, 0.0, 3, residual=x)).all()


# ------------------------------------------------------------ the sizes' ends, 32 bits

def _tiles_agree(t, rows, what):
    """Every block of `rows` rows holds the first one's bits."""
    t = t.view(-1, rows, t.shape[-1])
    for i in range(1, t.shape[0]):
        assert torch.equal(t[i], t[0]), f"{what}, block {i}"


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 99])
def test_layernorm_past_32_bits(C):
    """More than 2^31 elements: the same 2^16 rows again and again."""
    rows = 1 << 16
    n = (1 << 31) // (rows * C) + 2
    x, g, b, dy = _ln_rows(rows, C, "bf16", seed=C)
    X, D = x.repeat(n, 1), dy.repeat(n, 1)
    y, mean, rstd = cb.layernorm_forward(X, g, b, eps=1e-5, stats=True)
    cb.check_status()
    _ln_fwd_check(x, g, b, 1e-5, "bf16", y[:rows], mean[:rows], rstd[:rows], "first rows")
    for t, what in ((y, "y"), (mean[:, None], "mean"), (rstd[:, None], "rstd")):
        _tiles_agree(t, rows, what)
    dx, dg, db = cb.layernorm_backward(D, X, mean, rstd, g, out=D)
    cb.check_status()
    _ln_bwd_check(dy, x, g, mean[:rows], rstd[:rows], "bf16", (dx[:rows], None, None), "first rows")
    _tiles_agree(dx, rows, "dx")
    DY, N = dy.double(), (x.double() - mean[:rows, None].double()) * rstd[:rows, None].double()
    u = TYPES["bf16"][1]
    for got, terms in ((dg, DY * N), (db, DY)):     # chains of n rows / (296 blocks of 16 rows or more), 64 more
        chain = n * rows // (296 * 16) + 128
        _within(got, n * terms.sum(0), u * n * terms.sum(0).abs() + 1.01 * chain * E32 * n * terms.abs().sum(0), "columns")


@pytest.mark.gpu
def test_dropout_past_32_bits():
    """2^32 + 13 elements: their block numbers pass 2^29, their byte offsets 2^33."""
    n, seed, offset = (1 << 32) + 13, 77, 1 << 40
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = cb.dropout_forward(x, 0.25, seed, offset, out=x)
    cb.check_status()
    for at in (0, (1 << 31) - 4096, (1 << 32) - 4096, (n - 4096) // 8 * 8):
        m = min(8192, n - at)
        blocks = np.arange(at // 8, (at + m + 7) // 8, dtype=np.uint64)
        ctr = np.stack([blocks & np.uint64(0xFFFFFFFF), blocks >> np.uint64(32), np.full_like(blocks, offset & 0xFFFFFFFF),
                        np.full_like(blocks, offset >> 32)], axis=1)
        words = branch.philox(ctr, (seed, 0))
        draws = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], axis=2).reshape(-1)[:m]
        assert np.array_equal(tb.to64(y[at:at + m]) != 0, draws >= 16384), at


@pytest.mark.gpu
def test_gated_past_32_bits():
    """Z of more than 2^31 elements: the same 4096 rows again and again."""
    rows, n, C, F = 4096, 132, 8, 2048
    x, w, dh = tg._inputs(rows, C, F, "bf16", seed=4)
    X, D = x.repeat(n, 1), dh.repeat(n, 1)
    h, z = cb.gated_forward(X, w, preact=True)
    cb.check_status()
    assert z.numel() > 1 << 31
    tg._check_forward(x[:300], w, "silu", "bf16", h[:300], z[:300], "first rows")
    _tiles_agree(h, rows, "h")
    _tiles_agree(z, rows, "z")
    dx, dw = cb.gated_backward(D, X, z, w)
    cb.check_status()
    _tiles_agree(dx, rows, "dx")
    one = z[:rows].clone()
    DW = _dw64(dh, x, one)
    _check_gated_backward(dh, x, one, w, "bf16", dx[:rows], None, "first rows")
    u = HALF["bf16"][1]
    assert float((dw.double() - n * DW).norm() / (n * DW).norm()) <= 1.1 * (2 / 3) ** 0.5 * u


def _dw64(dh, x, z):
    DH, X, Z = _gpu64(dh, x, z)
    F = DH.shape[1]
    g, s = Z[:, :F], torch.sigmoid(Z[:, :F])
    return torch.cat([DH * Z[:, F:] * s * (1 + g * (1 - s)), DH * g * s], 1).t() @ X


# The widest blocks: C and F at their limits, on every kind of kernel.
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(HALF))
@pytest.mark.parametrize("shape", [(1, 65536, 8), (20, 65536, 8), (40, 65536, 136), (1, 16, 32768), (20, 16, 32768), (40, 72, 32768)],
                         ids=lambda s: "x".join(map(str, s)))
def test_gated_widest(shape, dtype):
    M, C, F = shape
    gen = torch.Generator(device="cuda").manual_seed(C + F)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    t, u, eta = HALF[dtype]
    x, w, dh = rnd(M, C).to(t), (1.5 * rnd(2 * F, C) / C ** 0.5).to(t), (0.3 * rnd(M, F)).to(t)
    h, z = cb.gated_forward(x, w, preact=True)
    cb.check_status()
    X, W = _gpu64(x, w)
    ref, d = X @ W.t(), C * E32 * (X.abs() @ W.abs().t())
    _within(z, ref, u * ref.abs() + (1 + u) * d + eta, "z")
    g, o, s = ref[:, :F], ref[:, F:], torch.sigmoid(ref[:, :F])
    e = 1.2 * o.abs() * d[:, :F] + (g * s).abs() * d[:, F:] + (25 + 4 * g.abs()) * E32 * (g * s * o).abs()
    _within(h, g * s * o, u * (g * s * o).abs() + (1 + u) * 1.01 * e + eta, "h")
    dx, dw = cb.gated_backward(dh, x, z, w)
    cb.check_status()
    _check_gated_backward(dh, x, z, w, dtype, dx, dw, "widest")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(3, 65536), (700, 65535), (2, 65533)], ids=lambda s: "x".join(map(str, s)))
def test_layernorm_widest(shape, dtype):
    _many(shape, dtype, "widest")


# ---------------------------------------------------------------- sums over splits

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(HALF))
@pytest.mark.parametrize("splits", [1, 2, 3, 4, 8, 9, 10, 16, 17, 18, 25, 32])
def test_every_split_is_added_once(splits, dtype):
    """Whole numbers: every split's partial is exact, and so is their sum."""
    gen = torch.Generator(device="cuda").manual_seed(splits)
    ints = lambda *s: torch.randint(-1, 2, s, generator=gen, device="cuda").to(HALF[dtype][0])
    K = 128 * splits               # two k-blocks of 64 to a split
    dy, w = ints(1, 1, 37, K), ints(K, 72)
    dy *= (torch.arange(K, device="cuda") % 64 < 4).to(dy.dtype)   # sums within 256, whole numbers in either type
    _, used = cb.splitk_workspace_bytes(1, 1, 37, K, 72, splits)
    got = cb.pointwise_splitk(dy, w, splits=splits)
    cb.check_status()
    assert used == splits
    want = dy.double().view(37, K) @ w.double()
    assert torch.equal(got.double().view(37, 72), want)


# --------------------------------------------------------------------- first calls

FIRST = """
import threading, torch, convolution_backward_b200 as cb
cases = []
for i in range(8):
    g = torch.Generator(device="cuda").manual_seed(i)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").half()
    M, C, F = 300 + 40 * i, 136, 264
    cases.append((r(M, F), r(M, C), r(M, 2 * F), r(2 * F, C) / 8))
torch.cuda.synchronize()
got, start = [None] * 8, threading.Barrier(8)
def work(i):
    s = torch.cuda.Stream()
    start.wait()
    got[i] = cb.gated_backward(*cases[i], stream=s)
    s.synchronize()
ts = [threading.Thread(target=work, args=(i,)) for i in range(8)]
[t.start() for t in ts]; [t.join() for t in ts]
for c, o in zip(cases, got):
    assert all(torch.equal(p, q) for p, q in zip(cb.gated_backward(*c), o))
cb.check_status()
print("first calls agree")
"""


@pytest.mark.gpu
def test_first_calls_from_many_threads():
    """A process whose first calls come from eight threads at once."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "agree" in r.stdout, r.stdout + r.stderr
