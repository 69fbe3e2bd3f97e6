"""Layer norm and dropout, forward and backward, against the fp64 oracle
(oracle/branch.py), and their refusals.

Tolerances, elementwise, from the arithmetic (u: the output type's half step
relative to the value, eta: half its smallest subnormal; e = 2^-24, one fp32
rounding; all sums fp32):
  layer norm     A sum of C terms is a chain of at most max(32, C/512) additions per
                 thread and at most 32 more across threads: K roundings of its terms'
                 magnitudes, K = max(32, C/512) + 32.  mean is thus off by at most
                 K e mean|x|, rstd relatively by (K/2 + 4) e (the sum of squares, the
                 division by C, + eps, the root, the reciprocal; the mean's own error
                 enters squared), and y by the propagated sum plus 3 roundings.
  its gradient   n and q carry 3 roundings; the two means K as above; the result
                 4 more.  A column sum over M rows chains at most M + 64 additions.
  dropout        the scale's rounding, the product-sum's, and the output's.
"""
import ctypes

import numpy as np
import pytest

import convolution_backward_b200 as cb
from oracle import branch

torch = pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, 1, 2, 3
FAKE = 0x10000000        # 16-byte aligned, never dereferenced
E32 = 2.0 ** -24
TYPES = {"f32": (torch.float32, 2.0 ** -24, 1e-30), "bf16": (torch.bfloat16, 2.0 ** -8, 1e-30),
         "f16": (torch.float16, 2.0 ** -11, 2.0 ** -25)}


def to64(t):
    return t.detach().double().cpu().numpy()


def within(got, ref, bound, what):
    got = to64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) / bound, 0)), ref.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, worst at {i}: got {got[i]!r}, "
                             f"want {ref[i]!r}, bound {np.broadcast_to(bound, ref.shape)[i]!r}")


def chain(C):
    return max(32, -(-C // 512)) + 32


# ------------------------------------------------------------------- the oracle

def test_philox_published_values():
    ones = np.full((1, 4), 0xFFFFFFFF)
    assert branch.philox(np.zeros((1, 4), dtype=np.int64), (0, 0))[0].tolist() == \
        [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert branch.philox(ones, (0xFFFFFFFF, 0xFFFFFFFF))[0].tolist() == \
        [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def _difference(f, a, i, h=1e-6):
    p, m = a.copy(), a.copy()
    p[i] += h
    m[i] -= h
    return (f(p) - f(m)) / (2 * h)


def test_oracle_layernorm_gradients_by_differences():
    r = np.random.default_rng(3)
    x, g, b, dy = r.normal(size=(5, 11)), r.normal(size=11), r.normal(size=11), r.normal(size=(5, 11))
    _, mean, rstd = branch.layernorm(x, g, b, 1e-5)
    dx, dg, db = branch.layernorm_backward(dy, x, g, mean, rstd)
    for i in [(0, 0), (2, 7), (4, 10)]:
        assert abs(_difference(lambda a: (branch.layernorm(a, g, b, 1e-5)[0] * dy).sum(), x, i) - dx[i]) < 1e-7
    for i in (0, 10):
        assert abs(_difference(lambda a: (branch.layernorm(x, a, b, 1e-5)[0] * dy).sum(), g, i) - dg[i]) < 1e-7
        assert abs(_difference(lambda a: (branch.layernorm(x, g, a, 1e-5)[0] * dy).sum(), b, i) - db[i]) < 1e-7


# ------------------------------------------------------------------ host checks

def _ln_fwd(M=4, C=16, dtype=1, eps=1e-5, X=FAKE, g=0, b=0, Y=2 * FAKE, mean=0, rstd=0):
    return cb.lib().dgrad_layernorm_forward(M, C, dtype, eps, X, g, b, Y, mean, rstd, None)


def test_layernorm_forward_refusals():
    assert _ln_fwd(M=-1) == INVALID
    assert _ln_fwd(C=0) == INVALID
    assert _ln_fwd(dtype=3) == INVALID
    assert _ln_fwd(eps=-1e-9) == INVALID
    assert _ln_fwd(eps=float("nan")) == INVALID
    assert _ln_fwd(eps=float("inf")) == INVALID
    assert _ln_fwd(eps=1e300) == INVALID            # infinite as fp32
    assert _ln_fwd(C=65537) == UNSUPPORTED
    assert _ln_fwd(M=1 << 31) == UNSUPPORTED
    assert _ln_fwd(X=0) == INVALID
    assert _ln_fwd(Y=0) == INVALID
    assert _ln_fwd(X=FAKE + 2) == ALIGNMENT
    assert _ln_fwd(g=FAKE + 8) == ALIGNMENT
    assert _ln_fwd(mean=FAKE + 2) == ALIGNMENT
    assert _ln_fwd(Y=FAKE + 16) == INVALID          # shifted over X
    assert _ln_fwd(g=2 * FAKE + 32) == INVALID      # gamma inside Y
    assert _ln_fwd(mean=3 * FAKE, rstd=3 * FAKE) == INVALID
    assert _ln_fwd(mean=FAKE) == INVALID
    assert _ln_fwd(M=0, X=0, Y=0) == OK


def _ln_bwd(M=4, C=16, dtype=1, dY=FAKE, X=2 * FAKE, g=0, mean=3 * FAKE, rstd=4 * FAKE, dX=5 * FAKE, dg=6 * FAKE,
            db=7 * FAKE, ws=8 * FAKE, nb=1 << 20):
    return cb.lib().dgrad_layernorm_backward(M, C, dtype, dY, X, g, mean, rstd, dX, dg, db, ws, nb, None)


def test_layernorm_backward_refusals():
    nb = ctypes.c_size_t(7)
    size = cb.lib().dgrad_layernorm_backward_workspace
    assert size(4, 16, 1, None) == INVALID
    assert size(0, 16, 1, ctypes.byref(nb)) == OK and nb.value == 0
    assert size(4, 0, 1, ctypes.byref(nb)) == INVALID
    assert size(4, 16, 1, ctypes.byref(nb)) == OK and nb.value > 0
    assert _ln_bwd(ws=0) == INVALID
    assert _ln_bwd(nb=nb.value - 1) == INVALID
    for name in ("dY", "X", "mean", "rstd", "dX"):
        assert _ln_bwd(**{name: 0}) == INVALID, name
    for name in ("dY", "X", "dX", "dg", "db", "ws"):
        assert _ln_bwd(**{name: 9 * FAKE + 8}) == ALIGNMENT, name
    assert _ln_bwd(rstd=4 * FAKE + 1) == ALIGNMENT
    assert _ln_bwd(dX=FAKE + 32) == INVALID
    assert _ln_bwd(dg=FAKE) == INVALID
    assert _ln_bwd(db=6 * FAKE) == INVALID
    assert _ln_bwd(ws=5 * FAKE) == INVALID
    assert _ln_bwd(mean=5 * FAKE) == INVALID
    assert _ln_bwd(M=0, dY=0, X=0, mean=0, rstd=0, dX=0, dg=0, db=0, ws=0, nb=0) == OK


def _drop(n=64, dtype=1, p=0.5, X=FAKE, r=0, Y=2 * FAKE):
    return cb.lib().dgrad_dropout_forward(n, dtype, p, 1, 2, X, r, Y, None)


def test_dropout_refusals():
    for p in (-0.1, 1.1, float("nan"), float("inf")):
        assert _drop(p=p) == INVALID
    assert _drop(n=-1) == INVALID
    assert _drop(n=(1 << 48) + 1) == UNSUPPORTED
    assert _drop(dtype=-1) == INVALID
    assert _drop(X=0) == INVALID
    assert _drop(Y=0) == INVALID
    assert _drop(X=FAKE + 4) == ALIGNMENT
    assert _drop(r=FAKE + 8) == ALIGNMENT
    assert _drop(Y=FAKE + 16) == INVALID
    assert _drop(r=2 * FAKE - 16) == INVALID
    assert _drop(n=0, X=0, Y=0) == OK
    assert cb.lib().dgrad_dropout_backward(64, 1, 0.5, 1, 2, FAKE, FAKE + 16, None) == INVALID


class _Fake:
    """A CUDA tensor's attributes, for checks that come before any library call."""

    def __init__(self, shape, dtype=torch.bfloat16, index=0, contiguous=True):
        self.shape, self.dtype, self.device, self.is_cuda = tuple(shape), dtype, torch.device("cuda", index), True
        self._c = contiguous

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return self._c

    def numel(self):
        return int(np.prod(self.shape))


def test_binding_refusals():
    x = _Fake((4, 16))
    with pytest.raises(ValueError, match="CUDA"):
        cb.layernorm_forward(torch.zeros(4, 16))
    with pytest.raises(ValueError, match="contiguous"):
        cb.layernorm_forward(_Fake((4, 16), contiguous=False))
    with pytest.raises(ValueError, match="gamma"):
        cb.layernorm_forward(x, _Fake((15,)))
    with pytest.raises(TypeError, match="beta"):
        cb.layernorm_forward(x, None, _Fake((16,), torch.float32))
    with pytest.raises(ValueError, match="same CUDA device"):
        cb.layernorm_forward(x, _Fake((16,), index=1))
    with pytest.raises(TypeError):
        cb.layernorm_forward(_Fake((4, 16), torch.float64))
    with pytest.raises(ValueError):
        cb.layernorm_forward(_Fake(()))
    with pytest.raises(ValueError, match="out"):
        cb.layernorm_forward(x, out=_Fake((4, 15)))
    s = _Fake((4,), torch.float32)
    with pytest.raises(ValueError, match="dY"):
        cb.layernorm_backward(_Fake((4, 15)), x, s, s)
    with pytest.raises(TypeError, match="mean"):
        cb.layernorm_backward(x, x, _Fake((4,)), s)
    with pytest.raises(ValueError, match="rstd"):
        cb.layernorm_backward(x, x, s, _Fake((4, 1), torch.float32))
    with pytest.raises(ValueError, match="residual"):
        cb.dropout_forward(x, 0.1, 1, residual=_Fake((16, 4)))
    for seed in (-1, 1 << 64):
        with pytest.raises(ValueError, match="seed"):
            cb.dropout_backward(x, 0.1, seed, out=x)
    with pytest.raises(TypeError):
        cb.layernorm_backward_workspace_bytes(4, 16, torch.int8)


# ------------------------------------------------------------------ layer norm

def _ln_inputs(M, C, dtype, seed, offset=0.5):
    r = np.random.default_rng(seed)
    t = TYPES[dtype][0]
    mk = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32)).to(t).cuda()
    x = mk(r.normal(size=(M, C)) * np.exp(0.4 * r.normal(size=C)) + offset * r.normal(size=C))
    return x, mk(1 + 0.2 * r.normal(size=C)), mk(0.2 * r.normal(size=C)), mk(r.normal(size=(M, C)))


def _check_fwd(x, g, b, eps, dtype, y, mean, rstd, what):
    C = x.shape[1]
    _, u, eta = TYPES[dtype]
    X = to64(x)
    G, B = (to64(g) if g is not None else np.ones(C)), (to64(b) if b is not None else np.zeros(C))
    ry, rm, rr = branch.layernorm(X, G, B, eps)
    K = chain(C)
    em = (K + 1) * E32 * np.abs(X).mean(axis=1) + E32 * np.abs(rm)
    # the mean's error shifts every difference: the sum of squares grows by C em^2
    er = ((K / 2 + 4) * E32 + 0.5 * (em * rr) ** 2) * rr
    within(mean, rm, em, what + " mean")
    within(rstd, rr, er, what + " rstd")
    n = (X - rm[:, None]) * rr[:, None]
    ey = ((em * rr)[:, None] + np.abs(n) * ((K / 2 + 8) * E32 + 0.5 * (em * rr)[:, None] ** 2)) * np.abs(G) \
        + 2 * E32 * (np.abs(n * G) + np.abs(B))
    within(y, ry, u * np.abs(ry) + (1 + u) * 1.01 * ey + eta, what + " y")


# sub-warp, one-warp and multi-warp rows, aligned and not, and rows too long for registers
LN_C = [1, 3, 7, 8, 13, 40, 57, 96, 100, 201, 384, 521, 768, 770, 1001, 1024, 1032, 1999, 2056, 2500, 4095, 5000, 5618,
        8197, 11111, 12296, 20001, 32776]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("C", LN_C)
def test_layernorm_forward(C, dtype):
    for M in (1, 37, 2530) if C < 2000 else (1, 5, 700):
        x, g, b, _ = _ln_inputs(M, C, dtype, seed=C + M)
        if C == 1:
            b = b + 1
        y, mean, rstd = cb.layernorm_forward(x, g, b, eps=1e-5, stats=True)
        _check_fwd(x, g, b, 1e-5, dtype, y, mean, rstd, f"M={M}")
        assert torch.equal(cb.layernorm_forward(x, g, b, eps=1e-5), y)
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("C", [96, 1001, 20001])
def test_layernorm_optional_parts(C, dtype):
    x, g, b, _ = _ln_inputs(9, C, dtype, seed=5)
    for gg, bb in ((None, None), (g, None), (None, b)):
        y, mean, rstd = cb.layernorm_forward(x, gg, bb, eps=1e-3, stats=True)
        _check_fwd(x, gg, bb, 1e-3, dtype, y, mean, rstd, f"gamma {gg is not None} beta {bb is not None}")
    want = cb.layernorm_forward(x, g, b)
    z = x.clone()
    assert cb.layernorm_forward(z, g, b, out=z) is z and torch.equal(z, want)   # in place
    x3 = x.view(3, 3, C)
    y3, m3, r3 = cb.layernorm_forward(x3, g, b, stats=True)
    assert y3.shape == x3.shape and m3.shape == (3, 3) and torch.equal(y3.view(9, C), want)


@pytest.mark.gpu
def test_layernorm_far_mean_and_odd_rows():
    """A mean far above the spread loses nothing to cancellation; a row with an infinity or
    NaN spoils only itself; a constant row gives beta."""
    x, g, b, _ = _ln_inputs(6, 768, "f32", seed=8)
    x = x + 3000.0
    y, mean, rstd = cb.layernorm_forward(x, g, b, eps=1e-5, stats=True)
    _check_fwd(x, g, b, 1e-5, "f32", y, mean, rstd, "far mean")
    clean = cb.layernorm_forward(x, g, b, eps=1e-5)
    x[1, 5], x[3, 700], x[4] = float("inf"), float("nan"), 2.5
    y = cb.layernorm_forward(x, g, b, eps=1e-5)
    assert torch.equal(y[[0, 2, 5]], clean[[0, 2, 5]])
    assert torch.isnan(y[1]).any() and torch.isnan(y[3]).all()
    assert torch.equal(y[4], b)


def _check_bwd(dy, x, g, mean, rstd, dtype, got, what):
    M, C = x.shape
    _, u, eta = TYPES[dtype]
    DY, X, m, r = to64(dy), to64(x), to64(mean), to64(rstd)
    G = to64(g) if g is not None else np.ones(C)
    dx, dg, db = branch.layernorm_backward(DY, X, G, m, r)
    n, q = (X - m[:, None]) * r[:, None], DY * G
    K = chain(C)
    aq, aqn = np.abs(q).mean(axis=1)[:, None], np.abs(q * n).mean(axis=1)[:, None]
    ex = r[:, None] * E32 * (5 * np.abs(q) + (K + 6) * aq + np.abs(n) * (K + 12) * aqn)
    within(got[0], dx, u * np.abs(dx) + (1 + u) * 1.01 * ex + eta, what + " dx")
    if got[1] is not None:
        k = (M + 64) * E32 * 1.01
        within(got[1], dg, u * np.abs(dg) + (1 + u) * (k + 3 * E32) * np.abs(DY * n).sum(axis=0) + eta, what + " dgamma")
        within(got[2], db, u * np.abs(db) + (1 + u) * k * np.abs(DY).sum(axis=0) + eta, what + " dbeta")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("C", LN_C)
def test_layernorm_backward(C, dtype):
    for M in (1, 37, 1200) if C < 2000 else (1, 5, 70, 700) if C < 6000 else (1, 5, 320):
        x, g, b, dy = _ln_inputs(M, C, dtype, seed=C + M)
        _, mean, rstd = cb.layernorm_forward(x, g, b, eps=1e-5, stats=True)
        got = cb.layernorm_backward(dy, x, mean, rstd, g)
        _check_bwd(dy, x, g, mean, rstd, dtype, got, f"M={M}")
        again = cb.layernorm_backward(dy, x, mean, rstd, g)
        assert all(torch.equal(a, c) for a, c in zip(got, again))
        only = cb.layernorm_backward(dy, x, mean, rstd, g, param_grads=False)
        assert only[1] is None and only[2] is None and torch.equal(only[0], got[0])
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("C", [96, 1001, 20001])
def test_layernorm_backward_variants(C, dtype):
    x, g, b, dy = _ln_inputs(50, C, dtype, seed=6)
    _, mean, rstd = cb.layernorm_forward(x, None, None, stats=True)
    got = cb.layernorm_backward(dy, x, mean, rstd)
    _check_bwd(dy, x, None, mean, rstd, dtype, got, "no gamma")
    want = cb.layernorm_backward(dy, x, mean, rstd, g)
    for which in (0, 1):        # dX written over dY, over X
        d, z = dy.clone(), x.clone()
        into = d if which == 0 else z
        got = cb.layernorm_backward(d, z, mean, rstd, g, out=into)
        assert got[0] is into and all(torch.equal(a, c) for a, c in zip(got, want))
    # a workspace of the stated size, what lies behind it left alone
    nb = cb.layernorm_backward_workspace_bytes(50, C, x.dtype)
    ws = torch.full((nb + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    got = cb.layernorm_backward(dy, x, mean, rstd, g, workspace=ws[:nb])
    assert all(torch.equal(a, c) for a, c in zip(got, want)) and bool((ws[nb:] == 0xA5).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(9000, 96), (7001, 201), (2500, 1001), (700, 4100)], ids=lambda s: "x".join(map(str, s)))
def test_layernorm_in_place_many_rows(shape, dtype):
    """Rows in flight for the next steps are not disturbed by results written over their tensor."""
    M, C = shape
    x, g, b, dy = _ln_inputs(M, C, dtype, seed=M)
    want = cb.layernorm_forward(x, g, b, stats=True)
    z = x.clone()
    got = cb.layernorm_forward(z, g, b, stats=True, out=z)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    grads = cb.layernorm_backward(dy, x, want[1], want[2], g)
    for which in (0, 1):
        d, z = dy.clone(), x.clone()
        got = cb.layernorm_backward(d, z, want[1], want[2], g, out=d if which == 0 else z)
        assert all(torch.equal(p, q) for p, q in zip(got, grads))
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 201, 4100, 20001])
def test_layernorm_c_calls_with_null_parts(C):
    """Either statistic and either parameter gradient alone."""
    M = 700
    x, g, b, dy = _ln_inputs(M, C, "bf16", seed=C)
    y, mean, rstd = cb.layernorm_forward(x, g, b, stats=True)
    dx, dg, db = cb.layernorm_backward(dy, x, mean, rstd, g)
    st = torch.cuda.current_stream().cuda_stream
    nb = cb.layernorm_backward_workspace_bytes(M, C, x.dtype)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    for which in (0, 1):
        o, stat, gr = torch.empty_like(y), torch.full_like(mean, 9.0), torch.empty_like(dg)
        p = [stat.data_ptr(), None] if which == 0 else [None, stat.data_ptr()]
        assert cb.lib().dgrad_layernorm_forward(M, C, 1, 1e-5, x.data_ptr(), g.data_ptr(), b.data_ptr(), o.data_ptr(), *p,
                                                st) == OK
        assert torch.equal(o, y) and torch.equal(stat, (mean, rstd)[which])
        p = [gr.data_ptr(), None] if which == 0 else [None, gr.data_ptr()]
        assert cb.lib().dgrad_layernorm_backward(M, C, 1, dy.data_ptr(), x.data_ptr(), g.data_ptr(), mean.data_ptr(),
                                                 rstd.data_ptr(), o.data_ptr(), *p, ws.data_ptr(), nb, st) == OK
        assert torch.equal(o, dx) and torch.equal(gr, (dg, db)[which])


@pytest.mark.gpu
def test_layernorm_gradient_by_differences():
    """Central differences of the fp32 forward along a direction v, step h = 2^-5, against <dX, v>.
    The step's own error is h^2/6 times the third derivative along v, below 40 in size here
    (|v| = 1 per element, the row's spread near 1, three powers of it and constants up to 6
    with sum(dY) weights of 1/sqrt(C)); the forward's rounding enters as 2e sqrt(M C)|y|/h."""
    M, C = 64, 384
    x, g, b, dy = _ln_inputs(M, C, "f32", seed=21, offset=0.0)
    x = x / x.std()
    v = torch.randn(M, C, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    h = 2.0 ** -5
    _, mean, rstd = cb.layernorm_forward(x, g, b, eps=1e-5, stats=True)
    dx, dg, db = cb.layernorm_backward(dy, x, mean, rstd, g)
    loss = lambda t, gg=g, bb=b: (cb.layernorm_forward(t, gg, bb, eps=1e-5).double() * dy.double()).sum()
    scale = float((dx.double() * v.double()).norm())
    assert abs(float((loss(x + h * v) - loss(x - h * v)) / (2 * h) - (dx.double() * v.double()).sum())) \
        <= 40 / 6 * h * h * scale + 4 * E32 * (M * C) ** 0.5 * 8 / h
    # the parameters enter linearly: only rounding is left
    w = v[0].contiguous()
    assert abs(float((loss(x, g + h * w) - loss(x, g - h * w)) / (2 * h) - (dg.double() * w.double()).sum())) \
        <= 4 * E32 * (M * C) ** 0.5 * 8 / h
    assert abs(float((loss(x, g, b + h * w) - loss(x, g, b - h * w)) / (2 * h) - (db.double() * w.double()).sum())) \
        <= 4 * E32 * (M * C) ** 0.5 * 8 / h


@pytest.mark.gpu
def test_layernorm_empty_and_edges():
    x = torch.empty(0, 24, device="cuda")
    s = torch.empty(0, device="cuda")
    g = torch.ones(24, device="cuda")
    assert cb.layernorm_forward(x, g).shape == (0, 24)
    dx, dg, db = cb.layernorm_backward(x, x, s, s, g)
    assert dx.shape == (0, 24) and not dg.any() and not db.any()
    # what lies behind the last row stays as it was
    buf = torch.full((8 * 40,), 7.0, device="cuda")
    cb.layernorm_forward(torch.randn(7, 40, device="cuda"), out=buf[:280].view(7, 40))
    assert bool((buf[280:] == 7).all())


# --------------------------------------------------------------------- dropout

def _check_drop(x, r, p, seed, offset, dtype, got, what):
    _, u, eta = TYPES[dtype]
    keep, scale = branch.dropout_keep(x.numel(), p, seed, offset)
    keep = keep.reshape(x.shape)
    X = np.where(keep, to64(x), 0.0)
    ref = X * scale + (to64(r) if r is not None else 0.0)
    e = E32 * (np.abs(X * scale) + np.abs(ref)) * 1.01
    within(got, ref, u * np.abs(ref) + (1 + u) * e + eta, what)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n", [1, 7, 8, 9, 4096, 100_003, 2_500_001])
def test_dropout(n, dtype):
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, generator=g, device="cuda").to(TYPES[dtype][0])
    r = torch.randn(n, generator=g, device="cuda").to(TYPES[dtype][0])
    seed, offset = 0xFEDCBA9876543210, (5 << 40) + n
    for p in (0.0, 0.1, 0.37, 1.0):
        for res in (None, r):
            _check_drop(x, res, p, seed, offset, dtype, cb.dropout_forward(x, p, seed, offset, residual=res),
                        f"p={p} residual={res is not None}")
    # the backward pass draws the same bits
    assert torch.equal(cb.dropout_backward(x, 0.37, seed, offset), cb.dropout_forward(x, 0.37, seed, offset))
    z = x.clone()
    assert torch.equal(cb.dropout_forward(z, 0.37, seed, offset, residual=z, out=z),
                       cb.dropout_forward(x, 0.37, seed, offset, residual=x))
    cb.check_status()


@pytest.mark.gpu
def test_dropout_leaves_no_trace_of_what_it_drops():
    x = torch.full((4096,), float("nan"), device="cuda", dtype=torch.bfloat16)
    keep, _ = branch.dropout_keep(4096, 0.5, 9, 1)
    y = cb.dropout_forward(x, 0.5, 9, 1)
    assert np.array_equal(np.isnan(to64(y)), keep) and not to64(y)[~keep].any()
    buf = torch.full((48,), 3.0, device="cuda")
    cb.dropout_backward(torch.randn(37, device="cuda"), 0.5, 1, out=buf[:37])
    assert bool((buf[37:] == 3).all())
    assert cb.dropout_forward(torch.empty(0, 8, device="cuda"), 0.5, 1).shape == (0, 8)


@pytest.mark.gpu
def test_dropout_rate():
    """Kept share and its spread over seeds: binomial, within 5 standard deviations."""
    n = 1 << 20
    x = torch.ones(n, device="cuda")
    for seed in range(4):
        kept = int((cb.dropout_forward(x, 0.3, seed) != 0).sum())
        assert abs(kept - 0.7 * n) < 5 * (n * 0.21) ** 0.5


# ------------------------------------------------- the debug build, streams, graphs

@pytest.fixture
def debug_library(monkeypatch):
    import os
    path = os.path.join(os.path.dirname(cb.library_path()), "libdgrad_debug.so")
    if not os.path.exists(path):
        pytest.skip("libdgrad_debug.so not built")
    monkeypatch.setattr(cb, "_LIB_PATH", path)
    monkeypatch.setattr(cb, "_lib", None)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(9, 13), (700, 96), (1500, 201), (1200, 770), (90, 4095), (3, 12296), (5, 32776)],
                         ids=lambda s: "x".join(map(str, s)))
def test_every_store_in_bounds(shape, dtype, debug_library):
    """The debug build checks every hand-indexed store against its buffer."""
    M, C = shape
    x, g, b, dy = _ln_inputs(M, C, dtype, seed=C)
    y, mean, rstd = cb.layernorm_forward(x, g, b, eps=1e-5, stats=True)
    got = cb.layernorm_backward(dy, x, mean, rstd, g)
    d = cb.dropout_forward(x, 0.3, 11, 2, residual=dy)
    cb.check_status()
    _check_fwd(x, g, b, 1e-5, dtype, y, mean, rstd, "debug")
    _check_bwd(dy, x, g, mean, rstd, dtype, got, "debug")
    _check_drop(x, dy, 0.3, 11, 2, dtype, d, "debug")


@pytest.mark.gpu
def test_two_calls_at_once():
    """The same operators on two streams at the same time, each with its own tensors."""
    a, b = _ln_inputs(5000, 768, "bf16", 1), _ln_inputs(3000, 1001, "f32", 2)

    def step(t, stream=None):
        x, g, be, dy = t
        y, m, r = cb.layernorm_forward(x, g, be, stats=True, stream=stream)
        z = cb.dropout_forward(y, 0.1, 3, 4, residual=x, stream=stream)
        return (z, *cb.layernorm_backward(dy, x, m, r, g, stream=stream))

    want = [[t.clone() for t in step(k)] for k in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = [step(k, s) for k, s in zip((a, b), streams)]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for o, w in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(o, w))
    cb.check_status()


@pytest.mark.gpu
def test_stream_of_another_device_is_refused():
    class Other:
        device = torch.device("cuda", 7)
        cuda_stream = 0

    with pytest.raises(ValueError, match="stream"):
        cb.layernorm_forward(torch.zeros(4, 8, device="cuda"), stream=Other())
    with pytest.raises(ValueError, match="stream"):
        cb.dropout_backward(torch.zeros(4, 8, device="cuda"), 0.1, 1, stream=Other())
