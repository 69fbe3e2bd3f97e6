"""Group norm with an activation, channels last, forward and backward, against the fp64 oracle
(oracle/branch.py), and its refusals.

Tolerances, elementwise, from the arithmetic (u: the output type's half step relative to the
value, eta: half its smallest subnormal; e = 2^-24; all sums fp32).  A sum over the S positions and
D channels of a group is formed by threads that add at most S values each, and joined over
threads and blocks in less than 128 additions more: K = S + 128 roundings of the terms' magnitudes.
  statistics  mean is off by (K + 4) e mean|x|.  Squares are summed about some mean of the group's own
              values, at most max|x - mean| from the mean: the sum is at most A = 1 + max n^2 times
              the one about the mean, so rstd is off relatively by A (K + 8) e / 2 + 4 e.
  z, act      n carries the statistics' errors and 3 roundings, z two more; the activation's error
              is test_branch_edges.act64's, and what z is off by enters it with the slope.
  gradients   dz: z's error times |act''| <= 1.2, act's, two roundings; sums as above, over the samples
              N S / 32 additions more at most.
The bounds grow with the longest chain, which rounding errors of either sign do not: results in
fp32 are held as a whole to 3e-6 of their norm besides.
"""
import ctypes

import numpy as np
import pytest

import convolution_backward_b200 as cb
import test_branch_edges as te
import test_branch_ops as tb
from oracle import branch

torch = pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, 1, 2, 3
FAKE = tb.FAKE
E32 = 2.0 ** -24
TYPES = tb.TYPES
ACTS = [None, "silu", "gelu", "gelu_tanh", "relu", "sigmoid"]
to64, within = tb.to64, tb.within


# ------------------------------------------------------------------- the oracle

def _difference(f, a, i, h=1e-6):
    p, m = a.copy(), a.copy()
    p[i] += h
    m[i] -= h
    return (f(p) - f(m)) / (2 * h)


@pytest.mark.parametrize("act", ACTS)
def test_oracle_gradients_by_differences(act):
    r = np.random.default_rng(11)
    N, S, C, G = 2, 5, 12, 3
    x, g, b, dy = r.normal(size=(N, S, C)), r.normal(size=C), r.normal(size=C), r.normal(size=(N, S, C))
    _, mean, rstd = branch.groupnorm(x, G, g, b, 1e-5, act)
    dx, dg, db = branch.groupnorm_backward(dy, x, g, b, mean, rstd, act)
    for i in [(0, 0, 0), (1, 2, 7), (1, 4, 11)]:
        want = _difference(lambda a: (branch.groupnorm(a, G, g, b, 1e-5, act)[0] * dy).sum(), x, i)
        assert abs(want - dx[i]) < 1e-6
    for i in (0, 11):
        assert abs(_difference(lambda a: (branch.groupnorm(x, G, a, b, 1e-5, act)[0] * dy).sum(), g, i) - dg[i]) < 1e-6
        assert abs(_difference(lambda a: (branch.groupnorm(x, G, g, a, 1e-5, act)[0] * dy).sum(), b, i) - db[i]) < 1e-6


def test_one_group_of_one_position_is_layer_norm():
    r = np.random.default_rng(1)
    x, g, b = r.normal(size=(4, 1, 10)), r.normal(size=10), r.normal(size=10)
    y, mean, rstd = branch.groupnorm(x, 1, g, b, 1e-5)
    want = branch.layernorm(x[:, 0], g, b, 1e-5)
    assert np.allclose(y[:, 0], want[0]) and np.allclose(mean[:, 0], want[1]) and np.allclose(rstd[:, 0], want[2])


# ------------------------------------------------------------------ host checks

def _fwd(N=2, S=4, C=16, G=4, dtype=1, eps=1e-5, act=5, X=FAKE, g=0, b=0, Y=2 * FAKE, mean=0, rstd=0, ws=8 * FAKE, nb=1 << 20):
    return cb.lib().dgrad_groupnorm_forward(N, S, C, G, dtype, eps, act, X, g, b, Y, mean, rstd, ws, nb, None)


def test_forward_refusals():
    size = cb.lib().dgrad_groupnorm_forward_workspace
    nb = ctypes.c_size_t(7)
    assert size(2, 4, 16, 4, 1, None) == INVALID
    assert size(0, 4, 16, 4, 1, ctypes.byref(nb)) == OK and nb.value == 0
    assert size(2, 4, 16, 5, 1, ctypes.byref(nb)) == INVALID
    assert size(2, 4, 16, 4, 1, ctypes.byref(nb)) == OK
    large = dict(N=1, S=1 << 20, C=8, G=1)      # one group of 2^23 values: sums over the whole GPU
    assert size(1, 1 << 20, 8, 1, 1, ctypes.byref(nb)) == OK and nb.value > 0
    for bad in ({"N": -1}, {"S": -1}, {"C": 0}, {"G": 0}, {"G": 3}, {"G": 32}, {"dtype": 3}, {"eps": -1e-9},
                {"eps": float("nan")}, {"eps": 1e300}, {"act": 6}, {"act": -1}, {"X": 0}, {"Y": 0}, {"ws": 0, **large},
                {"nb": nb.value - 1, **large}):
        assert _fwd(**bad) == INVALID, bad
    assert _fwd(C=65544, G=8) == UNSUPPORTED
    assert _fwd(N=1 << 20, S=1 << 12) == UNSUPPORTED
    assert _fwd(N=1 << 30, S=1, G=4) == UNSUPPORTED
    assert _fwd(N=1 << 62, S=1 << 62) == UNSUPPORTED
    for name in ("X", "Y", "g", "b", "ws"):
        assert _fwd(**{name: 9 * FAKE + 8}) == ALIGNMENT, name
    assert _fwd(mean=9 * FAKE + 2) == ALIGNMENT
    assert _fwd(Y=FAKE + 16) == INVALID          # shifted over X
    assert _fwd(g=2 * FAKE + 32) == INVALID      # gamma inside Y
    assert _fwd(mean=3 * FAKE, rstd=3 * FAKE) == INVALID
    assert _fwd(mean=FAKE) == INVALID
    large.update(X=0x40 * FAKE, Y=0x50 * FAKE)
    assert _fwd(ws=0x40 * FAKE + 16, **large) == INVALID
    assert _fwd(ws=0x50 * FAKE + 16, **large) == INVALID
    assert _fwd(mean=8 * FAKE, **large) == INVALID
    assert _fwd(N=0, X=0, Y=0, ws=0, nb=0) == OK
    assert _fwd(S=0, X=0, Y=0, ws=0, nb=0) == OK


def _bwd(N=2, S=4, C=16, G=4, dtype=1, act=0, dY=FAKE, X=2 * FAKE, g=0, b=0, mean=3 * FAKE, rstd=4 * FAKE, dX=5 * FAKE,
         dg=6 * FAKE, db=7 * FAKE, ws=8 * FAKE, nb=1 << 20):
    return cb.lib().dgrad_groupnorm_backward(N, S, C, G, dtype, act, dY, X, g, b, mean, rstd, dX, dg, db, ws, nb, None)


def test_backward_refusals():
    size = cb.lib().dgrad_groupnorm_backward_workspace
    nb = ctypes.c_size_t(7)
    assert size(2, 4, 16, 4, 3, ctypes.byref(nb)) == INVALID
    assert size(2, 0, 16, 4, 1, ctypes.byref(nb)) == OK and nb.value == 0
    assert size(2, 4, 16, 4, 1, ctypes.byref(nb)) == OK and nb.value > 0
    for bad in ({"G": 3}, {"act": 6}, {"ws": 0}, {"nb": nb.value - 1}, {"dY": 0}, {"X": 0}, {"mean": 0}, {"rstd": 0},
                {"dX": 0}, {"dX": FAKE + 32}, {"dg": FAKE}, {"db": 6 * FAKE}, {"ws": 5 * FAKE}, {"mean": 5 * FAKE},
                {"g": 5 * FAKE}, {"b": 6 * FAKE}):
        assert _bwd(**bad) == INVALID, bad
    for name in ("dY", "X", "g", "b", "dX", "dg", "db", "ws"):
        assert _bwd(**{name: 9 * FAKE + 8}) == ALIGNMENT, name
    assert _bwd(rstd=4 * FAKE + 1) == ALIGNMENT
    assert _bwd(N=0, dY=0, X=0, mean=0, rstd=0, dX=0, dg=0, db=0, ws=0, nb=0) == OK


def test_the_gated_block_takes_no_act_none():
    assert cb.lib().dgrad_gated_forward(4, 16, 16, 1, 5, FAKE, 2 * FAKE, 3 * FAKE, 0, None) == INVALID


def test_binding_refusals():
    x = tb._Fake((2, 3, 16))
    with pytest.raises(ValueError, match="CUDA"):
        cb.groupnorm_forward(torch.zeros(2, 3, 16), 4)
    with pytest.raises(ValueError, match="contiguous"):
        cb.groupnorm_forward(tb._Fake((2, 3, 16), contiguous=False), 4)
    for groups in (0, -4, 3, 32):
        with pytest.raises(ValueError, match="groups"):
            cb.groupnorm_forward(x, groups)
    with pytest.raises(ValueError, match="samples"):
        cb.groupnorm_forward(tb._Fake((16,)), 4)
    with pytest.raises(ValueError, match="gamma"):
        cb.groupnorm_forward(x, 4, tb._Fake((15,)))
    with pytest.raises(TypeError, match="beta"):
        cb.groupnorm_forward(x, 4, None, tb._Fake((16,), torch.float32))
    with pytest.raises(ValueError, match="activation"):
        cb.groupnorm_forward(x, 4, act="swish")
    with pytest.raises(ValueError, match="same CUDA device"):
        cb.groupnorm_forward(x, 4, tb._Fake((16,), index=1))
    with pytest.raises(ValueError, match="out"):
        cb.groupnorm_forward(x, 4, out=tb._Fake((2, 3, 8)))
    s = tb._Fake((2, 4), torch.float32)
    with pytest.raises(ValueError, match="dY"):
        cb.groupnorm_backward(tb._Fake((2, 3, 8)), x, s, s)
    with pytest.raises(ValueError, match="mean"):
        cb.groupnorm_backward(x, x, tb._Fake((2,), torch.float32), s)
    with pytest.raises(TypeError, match="rstd"):
        cb.groupnorm_backward(x, x, s, tb._Fake((2, 4)))
    with pytest.raises(ValueError, match="rstd"):
        cb.groupnorm_backward(x, x, s, tb._Fake((2, 8), torch.float32))
    with pytest.raises(TypeError):
        cb.groupnorm_backward_workspace_bytes(2, 3, 16, 4, torch.int8)


@pytest.fixture(params=["", "s", "c"], ids=["auto", "streaming", "cluster"])
def way(request, monkeypatch):
    """The library's own choice between its two ways, the streaming one everywhere, the cluster one wherever it fits."""
    monkeypatch.setenv("DGRAD_GN_WAY", request.param)
    cb._gn_workspace.cache_clear()
    yield request.param
    cb._gn_workspace.cache_clear()


# ------------------------------------------------------------------ forward

def _inputs(N, S, C, dtype, seed, offset=0.5):
    r = np.random.default_rng(seed)
    t = TYPES[dtype][0]
    mk = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32)).to(t).cuda()
    x = mk(r.normal(size=(N, S, C)) * np.exp(0.4 * r.normal(size=C)) + offset * r.normal(size=C) + 0.3 * r.normal(size=(N, 1, 1)))
    return x, mk(1 + 0.2 * r.normal(size=C)), mk(0.2 * r.normal(size=C)), mk(r.normal(size=(N, S, C)))


def _par(t, C, constant):
    return np.full(C, constant) if t is None else to64(t)


def _act_err(act, z):
    """(act, act', error of act, error of act') at z in fp32."""
    if act is None:
        return z, np.ones_like(z), 0 * z, 0 * z
    a, d, rel, ed = te.act64(act, z)
    return a, d, rel * np.abs(a) + te.TINY, ed + te.TINY


def _check_fwd(x, G, g, b, eps, act, dtype, y, mean, rstd, what, whole=True):
    N, S, C = x.shape
    _, u, eta = TYPES[dtype]
    X = to64(x)
    gm, bt = _par(g, C, 1.0), _par(b, C, 0.0)
    _, rm, rr = branch.groupnorm(X, G, gm, bt, eps)
    K = S + 128
    grp = np.abs(X).reshape(N, S, G, C // G)
    em = (K + 4) * E32 * grp.mean(axis=(1, 3))
    n = (X - branch._spread(rm, C)) * branch._spread(rr, C)
    A = 1 + np.square(n).reshape(N, S, G, C // G).max(axis=(1, 3))
    er = (A * (K + 8) / 2 + 4) * E32 + 0.5 * (em * rr) ** 2
    if mean is not None:
        within(mean, rm, em, what + " mean")
        within(rstd, rr, er * rr, what + " rstd")
    z = n * gm + bt
    shift = branch._spread(em * rr, C)
    ez = (shift + np.abs(n) * (branch._spread(er, C) + 4 * E32)) * np.abs(gm) * (1 + 2 * E32) + 3 * E32 * (np.abs(n * gm) + np.abs(bt))
    a, d, ea, _ = _act_err(act, z)
    err = ea + ez * (np.abs(d) + 1.2 * ez)
    within(y, a, u * np.abs(a) + (1 + u) * 1.01 * err + eta, what + " y")
    if whole and dtype == "f32" and S * C // G >= 64:
        assert np.linalg.norm(to64(y) - a) <= 3e-6 * np.linalg.norm(a), what


# (S, C, G): groups of one channel, of one value, wider than a vector, across vectors, one group of all;
# rows of 16-byte vectors and not; more channels than a block has columns
SHAPES = [(1, 8, 1), (1, 8, 8), (2, 8, 4), (1, 1, 1), (7, 3, 3), (5, 24, 8), (9, 30, 5), (49, 96, 32), (64, 512, 32), (37, 40, 1),
          (100, 129, 43), (33, 1001, 7), (300, 64, 16), (1000, 8, 2), (1111, 5, 1), (61, 2048, 32), (40, 2056, 8), (17, 4104, 2),
          (9, 4100, 50), (23, 520, 520), (2000, 320, 32)]
IDS = lambda s: "x".join(map(str, s))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(shape, dtype, way):
    S, C, G = shape
    for N, act in ((1, "silu"), (3, None), (17, "gelu")):
        x, g, b, _ = _inputs(N, S, C, dtype, seed=S + C + N)
        y, mean, rstd = cb.groupnorm_forward(x, G, g, b, eps=1e-5, act=act, stats=True)
        _check_fwd(x, G, g, b, 1e-5, act, dtype, y, mean, rstd, f"N={N} {act}")
        assert torch.equal(cb.groupnorm_forward(x, G, g, b, eps=1e-5, act=act), y)
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("act", ACTS)
def test_forward_activations_and_optional_parts(act, dtype, way):
    for S, C, G in ((50, 96, 8), (11, 33, 3)):
        x, g, b, _ = _inputs(4, S, C, dtype, seed=5)
        for gg, bb in ((None, None), (g, None), (None, b), (g, b)):
            y, mean, rstd = cb.groupnorm_forward(x, G, gg, bb, eps=1e-3, act=act, stats=True)
            _check_fwd(x, G, gg, bb, 1e-3, act, dtype, y, mean, rstd, f"gamma {gg is not None} beta {bb is not None}")
        z = x.clone()
        assert cb.groupnorm_forward(z, G, g, b, eps=1e-3, act=act, out=z) is z and torch.equal(z, y)     # in place
        y4 = cb.groupnorm_forward(x.view(4, S, 1, C), G, g, b, eps=1e-3, act=act)
        assert y4.shape == (4, S, 1, C) and torch.equal(y4.view(4, S, C), y)
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(400, 64, 8), (4000, 24, 1), (333, 21, 7)], ids=IDS)
def test_forward_far_mean_and_odd_rows(shape, way):
    """A mean far above the spread, a first position or block far from the others, constant groups, and
    an infinity or NaN, which spoil their own group alone."""
    S, C, G = shape
    x, g, b, _ = _inputs(3, S, C, "f32", seed=8)
    for change in ("far", "first", "half"):
        z = x + 3000.0
        if change == "first":
            z[:, 0] = 0.0
        if change == "half":
            z[:, S // 2:] -= 3500.0
        y, mean, rstd = cb.groupnorm_forward(z, G, g, b, stats=True)
        _check_fwd(z, G, g, b, 1e-5, None, "f32", y, mean, rstd, change, whole=False)   # fp32 holds 3000 to 2e-4
    clean = cb.groupnorm_forward(x, G, g, b, act="silu")
    D = C // G
    x[1, 3, 0], x[2, S - 1, C - 1] = float("inf"), float("nan")
    y, mean, rstd = cb.groupnorm_forward(x, G, g, b, act="silu", stats=True)
    assert torch.equal(y[0], clean[0])
    assert torch.isnan(y[1, :, :D]).all() and torch.equal(y[1, :, D:], clean[1, :, D:])
    assert torch.isnan(y[2, :, C - D:]).all() and torch.equal(y[2, :, :C - D], clean[2, :, :C - D])
    assert torch.isnan(rstd[1, 0]) and torch.isnan(mean[2, G - 1])
    const = torch.full((2, S, C), 2.5, device="cuda")
    y = cb.groupnorm_forward(const, G, g, b)
    assert torch.equal(y, b.expand_as(y))
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", [(60, 24, 8), (60, 32, 32), (50, 40, 8)], ids=IDS)
def test_nan_and_far_values_stay_in_their_group(shape, act, way):
    """Groups that end inside a 16-byte vector: a NaN, an infinity or a gamma that takes the activation to its ends in
    one of them changes nothing in the others."""
    S, C, G = shape
    D = C // G
    for dtype in TYPES:
        x, g, b, dy = _inputs(2, S, C, dtype, seed=S)
        y, mean, rstd = cb.groupnorm_forward(x, G, g, b, act=act, stats=True)
        grads = cb.groupnorm_backward(dy, x, mean, rstd, g, b, act=act)
        keep = torch.ones(C, dtype=torch.bool, device="cuda")
        keep[D:2 * D] = keep[3 * D:4 * D] = False
        for bad in (float("nan"), float("inf"), None):
            z, h = x.clone(), g.clone()
            if bad is None:
                h[~keep] = 6e4
            else:
                z[1, 7, D], z[0, 3, 3 * D] = bad, -bad
            y2, m2, r2 = cb.groupnorm_forward(z, G, h, b, act=act, stats=True)
            d2 = cb.groupnorm_backward(dy, z, m2, r2, h, b, act=act)
            assert torch.equal(y2[..., keep], y[..., keep]) and torch.equal(d2[0][..., keep], grads[0][..., keep])
            assert torch.equal(d2[1][keep], grads[1][keep]) and torch.equal(d2[2][keep], grads[2][keep])
            if bad is None and act in ("silu", "gelu", "gelu_tanh", "relu"):
                assert not (y2[..., ~keep] < -1).any() and torch.isfinite(y2.float()).any()
    cb.check_status()


@pytest.mark.gpu
def test_squares_past_the_range(way):
    """Values whose squares pass fp32's range: rstd 0, and beta is left; the other groups are untouched."""
    x, g, b, _ = _inputs(3, 300, 32, "f32", seed=4)
    clean = cb.groupnorm_forward(x, 4, g, b)
    x[1, :, :8] *= 1e25
    y, mean, rstd = cb.groupnorm_forward(x, 4, g, b, stats=True)
    assert torch.equal(y[1, :, :8], b[:8].expand(300, 8)) and rstd[1, 0] == 0 and torch.isfinite(mean).all()
    assert torch.equal(y[1, :, 8:], clean[1, :, 8:]) and torch.equal(y[0], clean[0])
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("C", [64, 61])
def test_two_streams_at_once(C, way):
    """Two calls that overlap, each with its own workspace, on streams of their own."""
    G = 8 if C == 64 else 61
    sets = [_inputs(6, 900, C, "bf16", seed=k) for k in (1, 2)]
    want = []
    for x, g, b, dy in sets:
        o = cb.groupnorm_forward(x, G, g, b, act="gelu", stats=True)
        want.append((*o, *cb.groupnorm_backward(dy, x, o[1], o[2], g, b, act="gelu")))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for (x, g, b, dy), s in zip(sets, streams):
            with torch.cuda.stream(s):
                o = cb.groupnorm_forward(x, G, g, b, act="gelu", stats=True)
                got.append((*o, *cb.groupnorm_backward(dy, x, o[1], o[2], g, b, act="gelu")))
        torch.cuda.synchronize()
        for w, q in zip(want, got):
            assert all(torch.equal(p, r) for p, r in zip(w, q))


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 99])
def test_past_32_bits(C):
    """More than 2^31 elements: the last samples against the same samples alone."""
    N, S = 34, -(-(1 << 31) // (33 * C))
    r = torch.Generator(device="cuda").manual_seed(1)
    few = torch.randn(2, S, C, device="cuda", generator=r).bfloat16()
    x = few.repeat(N // 2, 1, 1)
    assert x.numel() > 1 << 31
    g, b = torch.rand(C, device="cuda").bfloat16() + 0.5, torch.rand(C, device="cuda").bfloat16()
    y, mean, rstd = cb.groupnorm_forward(x, 3, g, b, act="silu", stats=True)
    assert all(torch.equal(y[k], y[k % 2]) for k in range(2, N))
    ref = branch.groupnorm(to64(few[1:, :, :]), 3, to64(g), to64(b), 1e-5, "silu")
    assert np.abs(to64(mean[N - 1]) - ref[1][0]).max() < 1e-4 and np.abs(to64(rstd[N - 1]) / ref[2][0] - 1).max() < 1e-4
    assert np.abs(to64(y[N - 1]) - ref[0][0]).max() <= 2.0 ** -8 * np.abs(ref[0]).max() + 1e-3
    dx, dg, db = cb.groupnorm_backward(y, x, mean, rstd, g, b, act="silu", out=y)
    assert all(torch.equal(dx[k], dx[k % 2]) for k in range(2, N))
    cb.check_status()


@pytest.mark.gpu
def test_no_samples_and_no_positions():
    g = torch.ones(8, device="cuda")
    for shape in ((0, 4, 8), (2, 0, 8), (2, 3, 0, 8)):
        x = torch.zeros(shape, device="cuda")
        y, mean, rstd = cb.groupnorm_forward(x, 2, g, g, stats=True)
        assert y.shape == x.shape and mean.shape == (shape[0], 2) and torch.isnan(mean).all() and torch.isnan(rstd).all()
        dx, dg, db = cb.groupnorm_backward(x, x, mean, rstd, g, g, act="silu")
        assert dx.shape == x.shape and not dg.any() and not db.any()
    cb.check_status()


# ------------------------------------------------------------------ backward

def _slope(act, x, g, b, mean, rstd):
    """(act'(z), its error): z in 64 bits, but for relu, whose border is defined in fp32 operations."""
    C = x.shape[2]
    gm, bt = _par(g, C, 1.0), _par(b, C, 0.0)
    n = (to64(x) - branch._spread(to64(mean), C)) * branch._spread(to64(rstd), C)
    z = n * gm + bt
    if act == "relu":
        f = lambda a: np.asarray(a, dtype=np.float32)
        z32 = ((f(to64(x)) - f(branch._spread(to64(mean), C))) * f(branch._spread(to64(rstd), C))) * f(gm) + f(bt)
        return n, (z32 > 0).astype(np.float64), 0 * z
    _, d, _, ed = _act_err(act, z)
    ez = 4 * E32 * (np.abs(n * gm) + np.abs(bt))
    return n, d, ed + (0 if act is None else 1.2 * ez)


def _check_bwd(dy, x, g, b, mean, rstd, act, dtype, got, what):
    N, S, C = x.shape
    G = mean.shape[1]
    _, u, eta = TYPES[dtype]
    DY, X, rs = to64(dy), to64(x), branch._spread(to64(rstd), C)
    gm, bt = _par(g, C, 1.0), _par(b, C, 0.0)
    n, slope, es = _slope(act, x, g, b, mean, rstd)
    dx, dg, db = branch.groupnorm_backward(DY, X, gm, bt, to64(mean), to64(rstd), act, slope)
    dz = DY * slope
    edz = np.abs(DY) * es + 2 * E32 * np.abs(dz)
    q, eq = dz * gm, np.abs(gm) * edz + E32 * np.abs(dz * gm)
    K = S + 160

    def mean_of(v):
        return branch._spread(v.reshape(N, S, G, C // G).mean(axis=(1, 3)), C)

    ea = mean_of(eq) + (K + 4) * E32 * mean_of(np.abs(q))
    eb = mean_of(eq * np.abs(n)) + (K + 8) * E32 * mean_of(np.abs(q * n))
    a, bb = mean_of(q), mean_of(q * n)
    ex = np.abs(rs) * (eq + ea + np.abs(n) * eb + 6 * E32 * (np.abs(q) + np.abs(a) + 2 * np.abs(n * bb)))
    within(got[0], dx, u * np.abs(dx) + (1 + u) * 1.01 * ex + eta, what + " dx")
    if got[1] is not None:
        K = S + 160 + N * S / 32
        en = edz * np.abs(n) + 4 * E32 * np.abs(dz * n)
        eg = en.sum(axis=(0, 1)) + K * E32 * np.abs(dz * n).sum(axis=(0, 1))
        within(got[1], dg, u * np.abs(dg) + (1 + u) * 1.01 * eg + eta, what + " dgamma")
        eB = edz.sum(axis=(0, 1)) + K * E32 * np.abs(dz).sum(axis=(0, 1))
        within(got[2], db, u * np.abs(db) + (1 + u) * 1.01 * eB + eta, what + " dbeta")
    if dtype == "f32" and S * C // G >= 64:
        assert np.linalg.norm(to64(got[0]) - dx) <= 3e-6 * np.linalg.norm(dx), what


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_backward(shape, dtype, way):
    S, C, G = shape
    for N, act in ((1, "silu"), (3, None), (17, "gelu")):
        x, g, b, dy = _inputs(N, S, C, dtype, seed=S + C + N)
        _, mean, rstd = cb.groupnorm_forward(x, G, g, b, eps=1e-5, act=act, stats=True)
        got = cb.groupnorm_backward(dy, x, mean, rstd, g, b, act=act)
        _check_bwd(dy, x, g, b, mean, rstd, act, dtype, got, f"N={N} {act}")
        again = cb.groupnorm_backward(dy, x, mean, rstd, g, b, act=act)
        assert all(torch.equal(p, q) for p, q in zip(got, again))
        only = cb.groupnorm_backward(dy, x, mean, rstd, g, b, act=act, param_grads=False)
        assert only[1] is None and only[2] is None and torch.equal(only[0], got[0])
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("act", ACTS)
def test_backward_activations_and_optional_parts(act, dtype, way):
    for S, C, G in ((50, 96, 8), (11, 33, 3)):
        x, g, b, dy = _inputs(4, S, C, dtype, seed=6)
        for gg, bb in ((None, None), (g, None), (None, b), (g, b)):
            _, mean, rstd = cb.groupnorm_forward(x, G, gg, bb, act=act, stats=True)
            got = cb.groupnorm_backward(dy, x, mean, rstd, gg, bb, act=act)
            _check_bwd(dy, x, gg, bb, mean, rstd, act, dtype, got, f"gamma {gg is not None} beta {bb is not None}")
        for which in (0, 1):        # dX written over dY, over X
            d, z = dy.clone(), x.clone()
            into = d if which == 0 else z
            again = cb.groupnorm_backward(d, z, mean, rstd, gg, bb, act=act, out=into)
            assert again[0] is into and all(torch.equal(p, q) for p, q in zip(got, again))
    cb.check_status()


@pytest.mark.gpu
def test_backward_of_groups_of_one_value_is_zero(way):
    x, g, b, dy = _inputs(5, 1, 24, "f32", seed=4)
    for act in ACTS:
        _, mean, rstd = cb.groupnorm_forward(x, 24, g, b, act=act, stats=True)
        assert torch.equal(mean, x[:, 0])
        dx, _, _ = cb.groupnorm_backward(dy, x, mean, rstd, g, b, act=act)
        assert not dx.any()


@pytest.mark.gpu
def test_gradients_by_differences_of_the_kernel():
    """fp32: the forward kernel's differences along random directions against the backward's products."""
    x, g, b, dy = _inputs(2, 30, 24, "f32", seed=9)
    r = np.random.default_rng(2)
    _, mean, rstd = cb.groupnorm_forward(x, 3, g, b, act="silu", stats=True)
    grads = cb.groupnorm_backward(dy, x, mean, rstd, g, b, act="silu")
    h = 1e-2
    for k, t in enumerate((x, g, b)):
        v = torch.from_numpy(r.normal(size=tuple(t.shape)).astype(np.float32)).cuda()
        ends = []
        for s in (h, -h):
            args = [x, g, b]
            args[k] = t + s * v
            y = cb.groupnorm_forward(args[0], 3, args[1], args[2], act="silu")
            ends.append((y.double() * dy.double()).sum().item())
        want = (grads[k].double() * v.double()).sum().item()
        # third derivatives times h^2/6: below 1e-3 of the terms' root-sum-square; fp32 sums far below
        scale = float((grads[k].double() ** 2).sum().sqrt() * (v.double() ** 2).sum().sqrt())
        assert abs((ends[0] - ends[1]) / (2 * h) - want) <= 3e-3 * scale


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(9, 50, 96, 8), (3, 33, 1001, 7), (2, 17, 4104, 2), (40, 1, 24, 24)], ids=IDS)
def test_every_store_in_bounds(shape, dtype, monkeypatch, way):
    """Under the debug build, whose stores check their place."""
    import os
    path = os.path.join(os.path.dirname(cb.library_path()), "libdgrad_debug.so")
    if not os.path.exists(path):
        pytest.skip("libdgrad_debug.so not built")
    monkeypatch.setattr(cb, "_LIB_PATH", path)
    monkeypatch.setattr(cb, "_lib", None)
    N, S, C, G = shape
    x, g, b, dy = _inputs(N, S, C, dtype, seed=3)
    y, mean, rstd = cb.groupnorm_forward(x, G, g, b, act="silu", stats=True)
    _check_fwd(x, G, g, b, 1e-5, "silu", dtype, y, mean, rstd, "debug")
    got = cb.groupnorm_backward(dy, x, mean, rstd, g, b, act="silu")
    _check_bwd(dy, x, g, b, mean, rstd, "silu", dtype, got, "debug")
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cluster", [1, 2, 4, 8])
@pytest.mark.parametrize("shape", [(3, 700, 96, 8, 2), (2, 1000, 40, 1, 1), (1, 4001, 66, 6, 3), (5, 9, 256, 32, 5), (2, 6000, 24, 8, 1)], ids=IDS)
def test_cluster_sizes(shape, cluster, dtype, monkeypatch):
    """Every cluster size; slices of unequal width; blocks without positions; more positions than fit the
    shared memory."""
    N, S, C, G, slices = shape
    monkeypatch.setenv("DGRAD_GN_WAY", "c")
    monkeypatch.setenv("DGRAD_GN_CLUSTER", str(cluster))
    monkeypatch.setenv("DGRAD_GN_SLICES", str(slices))
    cb._gn_workspace.cache_clear()
    x, g, b, dy = _inputs(N, S, C, dtype, seed=S + cluster)
    y, mean, rstd = cb.groupnorm_forward(x, G, g, b, act="silu", stats=True)
    _check_fwd(x, G, g, b, 1e-5, "silu", dtype, y, mean, rstd, "forward")
    got = cb.groupnorm_backward(dy, x, mean, rstd, g, b, act="silu")
    _check_bwd(dy, x, g, b, mean, rstd, "silu", dtype, got, "backward")
    cb.check_status()
    cb._gn_workspace.cache_clear()


@pytest.mark.gpu
def test_captured_streams_and_workspaces(way):
    """One workspace in two captured graphs, another stream, and a replay on new inputs."""
    N, S, C, G = 4, 200, 96, 8
    x, g, b, dy = _inputs(N, S, C, "bf16", seed=12)
    nb = max(cb.groupnorm_forward_workspace_bytes(N, S, C, G, x.dtype), cb.groupnorm_backward_workspace_bytes(N, S, C, G, x.dtype))
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    want = cb.groupnorm_forward(x, G, g, b, act="silu", stats=True)
    wgrad = cb.groupnorm_backward(dy, x, want[1], want[2], g, b, act="silu")
    graphs, outs = [], []
    for k in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = cb.groupnorm_forward(x, G, g, b, act="silu", stats=True, workspace=ws)
            d = cb.groupnorm_backward(dy, x, o[1], o[2], g, b, act="silu", workspace=ws)
        graphs.append(graph)
        outs.append((*o, *d))
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(p, q) for p, q in zip(out, (*want, *wgrad)))
    x2, _, _, _ = _inputs(N, S, C, "bf16", seed=13)
    w2 = cb.groupnorm_forward(x2, G, g, b, act="silu")
    x.copy_(x2)
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1][0], w2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = cb.groupnorm_forward(x2, G, g, b, act="silu", stream=side)
    side.synchronize()
    assert torch.equal(y, w2)
    with pytest.raises(cb.DgradError):
        cb.groupnorm_backward(dy, x, want[1], want[2], g, b, workspace=ws[:16])
