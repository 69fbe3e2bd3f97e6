"""The gated pointwise block, forward and backward, against the fp64 oracle
(oracle/branch.py), its refusals, and a whole residual branch of the operators together.

Tolerances, elementwise (u, eta: the output type's half step and half its smallest
subnormal; e = 2^-24):
  Z   fp32 accumulation of C products in any order: C e sum|x w|, then one rounding.
  H   g and u carry Z's fp32 error d; act is Lipschitz with constant 1.2, so
      |h| moves by 1.2 |u| d_g + |act(g)| d_u; act itself is off relatively by
      rel(g) = (10 + 4 max(|g|, g^2, |v|)) 2^-23: a few units for the quotient and the
      product, the fast exponential's error growing with its argument (|g|; 2|v| in
      the tanh form, v = sqrt(2/pi)(|g| + 0.044715|g|^3)), erfc's with twice its
      argument squared.  Then one rounding.
  dZ  the same, the derivative's terms summing to at most 1.5 in magnitude, and one
      rounding to the operand type; dX and dW sum it: err_dZ |W| + 2F e |dZ||W|,
      |err_dZ|^T |X| + M e |dZ|^T |X|, then one rounding.
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
TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8, 1e-30), "f16": (torch.float16, 2.0 ** -11, 2.0 ** -25)}
ACTS = list(cb.ACTIVATIONS)


def to64(t):
    return t.detach().double().cpu().numpy()


def within(got, ref, bound, what):
    got = to64(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) / bound, 0)), ref.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, worst at {i}: got {got[i]!r}, "
                             f"want {ref[i]!r}, bound {np.broadcast_to(bound, ref.shape)[i]!r}")


def act_rel(g):
    a = np.abs(g)
    v = 0.8 * (a + 0.044715 * a ** 3)
    return (10 + 4 * np.maximum(np.maximum(a, a * a), v)) * 2.0 ** -23


# ------------------------------------------------------------------- the oracle

@pytest.mark.parametrize("act", ACTS)
def test_oracle_gradients_by_differences(act):
    r = np.random.default_rng(4)
    x, w, dh = r.normal(size=(3, 5)), r.normal(size=(8, 5)), r.normal(size=(3, 4))
    z = branch.gated(x, w, act)[1]
    dx, dw = branch.gated_backward(dh, x, z, w, act)

    def loss(x, w):
        return (branch.gated(x, w, act)[0] * dh).sum()

    h = 1e-6
    for i in [(0, 0), (2, 4), (1, 2)]:
        e = np.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for i in [(0, 0), (3, 4), (4, 1), (7, 2)]:
        e = np.zeros_like(w)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


# ------------------------------------------------------------------ host checks

def _fwd(M=16, C=64, F=32, dtype=1, act=0, X=FAKE, W=2 * FAKE, H=3 * FAKE, Z=0):
    return cb.lib().dgrad_gated_forward(M, C, F, dtype, act, X, W, H, Z, None)


def test_forward_refusals():
    assert _fwd(dtype=0) == UNSUPPORTED
    assert _fwd(dtype=9) == INVALID
    assert _fwd(act=5) == INVALID
    assert _fwd(act=-1) == INVALID
    assert _fwd(M=-1) == INVALID
    assert _fwd(F=0) == INVALID
    assert _fwd(C=0) == INVALID
    assert _fwd(C=65544) == UNSUPPORTED
    assert _fwd(F=32776) == UNSUPPORTED
    assert _fwd(M=(1 << 30) + 1) == UNSUPPORTED
    assert _fwd(C=60) == ALIGNMENT
    assert _fwd(F=36) == ALIGNMENT
    for name in ("X", "W", "H"):
        assert _fwd(**{name: 0}) == INVALID, name
        assert _fwd(**{name: 7 * FAKE + 8}) == ALIGNMENT, name
    assert _fwd(Z=5 * FAKE + 2) == ALIGNMENT
    assert _fwd(H=FAKE) == INVALID
    assert _fwd(Z=3 * FAKE + 16) == INVALID
    assert _fwd(Z=2 * FAKE) == INVALID
    assert _fwd(M=0, X=0, W=0, H=0) == OK


def _bwd(M=16, C=64, F=32, dtype=1, act=0, dH=FAKE, X=2 * FAKE, Z=3 * FAKE, W=4 * FAKE, dX=5 * FAKE, dW=6 * FAKE,
         ws=7 * FAKE, nb=1 << 24):
    return cb.lib().dgrad_gated_backward(M, C, F, dtype, act, dH, X, Z, W, dX, dW, ws, nb, None)


def test_backward_refusals():
    nb = ctypes.c_size_t()
    size = cb.lib().dgrad_gated_backward_workspace
    assert size(16, 64, 32, None) == INVALID
    assert size(16, 60, 32, ctypes.byref(nb)) == ALIGNMENT
    assert size(0, 64, 32, ctypes.byref(nb)) == OK and nb.value == 0
    assert size(16, 64, 32, ctypes.byref(nb)) == OK and nb.value == 16 * 64 * 4        # few values: fp32 dZ
    assert size(1600, 64, 32, ctypes.byref(nb)) == OK and nb.value >= 1600 * 64 * 2
    assert size(16, 64, 32, ctypes.byref(nb)) == OK
    assert _bwd(dtype=0) == UNSUPPORTED
    assert _bwd(act=7) == INVALID
    assert _bwd(dX=0, dW=0) == INVALID
    assert _bwd(nb=nb.value - 1) == INVALID
    assert _bwd(ws=0) == INVALID
    for name in ("dH", "X", "Z", "W"):
        assert _bwd(**{name: 0}) == INVALID, name
    for name in ("dH", "X", "Z", "W", "dX", "dW", "ws"):
        assert _bwd(**{name: 9 * FAKE + 8}) == ALIGNMENT, name
    for a, b in (("dX", 2 * FAKE), ("dW", 4 * FAKE), ("ws", 3 * FAKE), ("dX", 6 * FAKE), ("ws", 5 * FAKE), ("dX", FAKE)):
        assert _bwd(**{a: b}) == INVALID, (a, b)
    assert _bwd(M=0, dX=0, dH=0, X=0, Z=0, W=0, ws=0, nb=0, dW=0) == INVALID
    assert _bwd(M=0, dW=0, dH=0, X=0, Z=0, W=0, ws=0, nb=0) == OK


class _Fake:
    def __init__(self, shape, dtype=torch.bfloat16, index=0):
        self.shape, self.dtype, self.device, self.is_cuda = tuple(shape), dtype, torch.device("cuda", index), True

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True


def test_binding_refusals():
    x, w = _Fake((4, 16)), _Fake((16, 16))
    with pytest.raises(ValueError, match="CUDA"):
        cb.gated_forward(torch.zeros(4, 16), torch.zeros(16, 16))
    with pytest.raises(ValueError, match="activation"):
        cb.gated_forward(x, w, act="swish")
    for bad in ((16, 15), (15, 16), (0, 16), (16,)):
        with pytest.raises(ValueError, match="W"):
            cb.gated_forward(x, _Fake(bad))
    with pytest.raises(TypeError, match="W"):
        cb.gated_forward(x, _Fake((16, 16), torch.float16))
    with pytest.raises(ValueError, match="same CUDA device"):
        cb.gated_forward(x, _Fake((16, 16), index=1))
    with pytest.raises(ValueError, match="out"):
        cb.gated_forward(x, w, out=_Fake((4, 16)))
    with pytest.raises(ValueError, match="dH"):
        cb.gated_backward(_Fake((4, 16)), x, _Fake((4, 16)), w)
    with pytest.raises(ValueError, match="Z"):
        cb.gated_backward(_Fake((4, 8)), x, _Fake((4, 8)), w)
    with pytest.raises(ValueError, match="nothing"):
        cb.gated_backward(_Fake((4, 8)), x, _Fake((4, 16)), w, input_grad=False, weight_grad=False)


# --------------------------------------------------------------------- forward

def _inputs(M, C, F, dtype, seed, gain=1.5):
    r = np.random.default_rng(seed)
    mk = lambda a: torch.from_numpy(a.astype(np.float32)).to(TYPES[dtype][0]).cuda()
    return (mk(r.normal(size=(M, C))), mk(gain * r.normal(size=(2 * F, C)) / C ** 0.5), mk(0.3 * r.normal(size=(M, F))))


def _check_forward(x, w, act, dtype, h, z, what):
    _, u, eta = TYPES[dtype]
    X, W = to64(x), to64(w)
    F, C = W.shape[0] // 2, W.shape[1]
    rh, rz = branch.gated(X, W, act)
    d = C * E32 * (np.abs(X) @ np.abs(W).T)
    if z is not None:
        within(z, rz, u * np.abs(rz) + (1 + u) * d + eta, what + " z")
    g, uu = rz[:, :F], rz[:, F:]
    a = branch.act(act, g)[0]
    eh = 1.2 * np.abs(uu) * d[:, :F] + np.abs(a) * d[:, F:] + np.abs(rh) * act_rel(g)
    within(h, rh, u * np.abs(rh) + (1 + u) * 1.01 * eh + eta, what + " h")


# rows kernels (up to 32 rows), narrow and wide tiles, ragged everywhere, more tiles than pairs
SHAPES = [(1, 8, 8), (1, 768, 264), (2, 264, 8), (3, 72, 40), (8, 136, 72), (9, 8, 8), (16, 520, 24), (25, 776, 104),
          (32, 40, 16), (33, 64, 48), (37, 72, 1000), (128, 64, 64),
          (257, 328, 264), (700, 200, 136), (2600, 136, 520), (5900, 72, 600)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, dtype):
    M, C, F = shape
    x, w, _ = _inputs(M, C, F, dtype, seed=M + C + F)
    for act in ACTS if M < 1000 else ("silu",):
        h, z = cb.gated_forward(x, w, act=act, preact=True)
        cb.check_status()
        _check_forward(x, w, act, dtype, h, z, act)
        assert torch.equal(cb.gated_forward(x, w, act=act), h), act
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_forward_large_arguments(act):
    """Gates far out on both sides: the activation's tails, no infinity from a finite result."""
    x, w, _ = _inputs(64, 64, 64, "bf16", seed=2, gain=40.0)
    h, z = cb.gated_forward(x, w, act=act, preact=True)
    assert torch.isfinite(h).all()
    g, u = to64(z)[:, :64], to64(z)[:, 64:]
    if act != "sigmoid":
        assert (np.abs(to64(h))[g < -30] <= 1e-8 * np.abs(u[g < -30])).all()


@pytest.mark.gpu
def test_forward_shapes_and_bounds():
    x, w, _ = _inputs(30, 64, 72, "bf16", seed=3)
    want = cb.gated_forward(x, w)
    got, z = cb.gated_forward(x.view(2, 3, 5, 64), w, preact=True)
    assert got.shape == (2, 3, 5, 72) and z.shape == (2, 3, 5, 144) and torch.equal(got.view(30, 72), want)
    for M in (4, 30):       # what lies behind the last row stays as it was
        buf = torch.full((M * 72 + 256,), 5.0, dtype=torch.bfloat16, device="cuda")
        cb.gated_forward(x[:M], w, out=buf[:M * 72].view(M, 72))
        assert bool((buf[M * 72:] == 5).all())
    assert cb.gated_forward(x[:0], w).shape == (0, 72)
    # rows do not mix: a NaN spoils its own
    x2 = x.clone()
    x2[7] = float("nan")
    got = cb.gated_forward(x2, w)
    keep = [i for i in range(30) if i != 7]
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[7]).all()


# -------------------------------------------------------------------- backward

def _check_backward(dh, x, z, w, act, dtype, dx, dw, what):
    _, u, eta = TYPES[dtype]
    DH, X, Z, W = to64(dh), to64(x), to64(z), to64(w)
    M, F = DH.shape
    dz = branch.gated_dz(DH, Z, act)
    g, uu = Z[:, :F], Z[:, F:]
    rel, a = act_rel(g), np.abs(branch.act(act, g)[0])
    e = u * np.abs(dz) + 1.01 * np.concatenate([1.5 * rel * np.abs(DH * uu), rel * np.abs(DH) * a], axis=1) + eta
    if dx is not None:
        ref = dz @ W
        within(dx, ref, u * np.abs(ref) + (1 + u) * (e @ np.abs(W) + 2 * F * E32 * 1.01 * (np.abs(dz) @ np.abs(W))) + eta,
               what + " dx")
    if dw is not None:
        ref = dz.T @ X
        within(dw, ref, u * np.abs(ref) + (1 + u) * (e.T @ np.abs(X) + M * E32 * 1.01 * (np.abs(dz).T @ np.abs(X))) + eta,
               what + " dw")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES + [(300, 1096, 1208), (4000, 264, 40), (1, 2048, 2048), (1, 520, 2056), (2, 72, 1024), (250, 200, 8), (256, 64, 8),
                                            (257, 64, 8), (512, 64, 8), (513, 64, 8)], ids=lambda s: "x".join(map(str, s)))
def test_backward(shape, dtype):
    M, C, F = shape
    x, w, dh = _inputs(M, C, F, dtype, seed=M + C + F + 1)
    for act in ACTS if M * F < 300_000 else ("silu",):
        z = cb.gated_forward(x, w, act=act, preact=True)[1]
        dx, dw = cb.gated_backward(dh, x, z, w, act=act)
        cb.check_status()
        _check_backward(dh, x, z, w, act, dtype, dx, dw, act)
        again = cb.gated_backward(dh, x, z, w, act=act)
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
        if act == "silu":
            only = cb.gated_backward(dh, x, z, w, act=act, weight_grad=False)
            assert only[1] is None and torch.equal(only[0], dx)
            only = cb.gated_backward(dh, x, z, w, act=act, input_grad=False)
            assert only[0] is None and torch.equal(only[1], dw)
    cb.check_status()


@pytest.mark.gpu
def test_backward_workspace_and_empty():
    x, w, dh = _inputs(1000, 136, 72, "bf16", seed=9)
    z = cb.gated_forward(x, w, preact=True)[1]
    want = cb.gated_backward(dh, x, z, w)
    nb = cb.gated_backward_workspace_bytes(1000, 136, 72)
    ws = torch.full((nb + 256,), 0xA5, dtype=torch.uint8, device="cuda")   # any contents: NaN patterns among them
    ws[:nb] = 0xFF
    got = cb.gated_backward(dh, x, z, w, workspace=ws[:nb])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and bool((ws[nb:] == 0xA5).all())
    dx, dw = cb.gated_backward(dh[:0], x[:0], z[:0], w)
    assert dx.shape == (0, 136) and dw.shape == w.shape and not dw.any()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(16, 72, 40), (900, 136, 72)], ids=lambda s: "x".join(map(str, s)))
def test_c_calls_with_null_parts(shape):
    """X may be null where dW is not wanted, W where dX is not."""
    M, C, F = shape
    x, w, dh = _inputs(M, C, F, "bf16", seed=3)
    z = cb.gated_forward(x, w, preact=True)[1]
    dx, dw = cb.gated_backward(dh, x, z, w)
    nb = cb.gated_backward_workspace_bytes(M, C, F)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    gx, gw = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
    call = lambda X, W, dX, dW: cb.lib().dgrad_gated_backward(M, C, F, 1, 0, dh.data_ptr(), X, z.data_ptr(), W, dX, dW,
                                                              ws.data_ptr(), nb, torch.cuda.current_stream().cuda_stream)
    assert call(None, w.data_ptr(), gx.data_ptr(), None) == OK
    assert call(x.data_ptr(), None, None, gw.data_ptr()) == OK
    assert torch.equal(gx, dx) and torch.equal(gw, dw)
    assert call(None, w.data_ptr(), gx.data_ptr(), gw.data_ptr()) == INVALID
    assert call(x.data_ptr(), None, gx.data_ptr(), gw.data_ptr()) == INVALID


@pytest.mark.gpu
def test_one_workspace_in_two_graphs():
    """Two captured backward passes of different sizes that share a workspace, replayed in turn."""
    cases = [_inputs(1500, 136, 264, "bf16", seed=1), _inputs(90, 264, 40, "f16", seed=2)]
    zs = [cb.gated_forward(x, w, preact=True)[1] for x, w, _ in cases]
    want = [[t.clone() for t in cb.gated_backward(dh, x, z, w)] for (x, w, dh), z in zip(cases, zs)]
    nb = max(cb.gated_backward_workspace_bytes(x.shape[0], x.shape[1], w.shape[0] // 2) for x, w, _ in cases)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for (x, w, dh), z in zip(cases, zs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(cb.gated_backward(dh, x, z, w, workspace=ws))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    for o, wv in zip(outs, want):
        assert all(torch.equal(p, q) for p, q in zip(o, wv))
    cb.check_status()


# ------------------------------------------------------------- the whole branch

class Branch:
    """y = x + dropout(down(gated(layernorm(x)))) and its gradients, from this package's calls.
    The down projection is a pointwise product: its forward takes the weight as (F, C), its
    gradient (dgrad) as (C, F)."""

    def __init__(self, M, C, F, dtype, seed):
        r = np.random.default_rng(seed)
        mk = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32)).to(TYPES[dtype][0]).cuda()
        self.x, self.dy = mk(r.normal(size=(1, 1, M, C))), mk(0.5 * r.normal(size=(1, 1, M, C)))
        self.gamma, self.beta = mk(1 + 0.1 * r.normal(size=C)), mk(0.1 * r.normal(size=C))
        self.w = mk(1.5 * r.normal(size=(2 * F, C)) / C ** 0.5)
        self.down = mk(r.normal(size=(F, C)) / F ** 0.5)
        self.down_t = self.down.t().contiguous()

    def forward_backward(self, stream=None):
        st = dict(stream=stream)
        n, mean, rstd = cb.layernorm_forward(self.x, self.gamma, self.beta, eps=1e-5, stats=True, **st)
        h, z = cb.gated_forward(n, self.w, preact=True, **st)
        d = cb.pointwise(h, self.down, **st)
        y = cb.dropout_forward(d, 0.2, 77, 5, residual=self.x, **st)
        dd = cb.dropout_backward(self.dy, 0.2, 77, 5, **st)
        dh = cb.pointwise(dd, self.down_t, **st)
        dn, dw = cb.gated_backward(dh, n, z, self.w, **st)
        dx, dg, db = cb.layernorm_backward(dn, self.x, mean, rstd, self.gamma, **st)
        return y, dx, dg, db, dw


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(300, 136, 264), (5, 64, 72)], ids=["300x136x264", "5x64x72"])
def test_branch_together(shape, dtype):
    """Against the same branch in fp64 with autograd.  Every 16-bit result rounds by u and the
    errors of a chain of at most seven of them add in norm: 7 sqrt(u^2/3) < 5 u of the result's
    norm, whose terms do not cancel (the residual and the branch are independent); 8 u allowed."""
    M, C, F = shape
    b = Branch(M, C, F, dtype, seed=1)
    y, dx, dg, db, dw = b.forward_backward()
    cb.check_status()
    x, g, be, w = (t.detach().double().requires_grad_() for t in (b.x, b.gamma, b.beta, b.w))
    mean = x.mean(-1, keepdim=True)
    n = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + 1e-5) * g + be
    z = n @ w.t()
    d = (z[..., :F] * torch.sigmoid(z[..., :F]) * z[..., F:]) @ b.down.double()
    keep, scale = branch.dropout_keep(M * C, 0.2, 77, 5)
    ref = x + d * torch.from_numpy(keep).cuda().view(d.shape) * scale
    ref.backward(b.dy.double())     # the residual passes dY on: layernorm_backward gives the rest
    u = TYPES[dtype][1]
    for name, got, want in (("y", y, ref), ("dx", dx, x.grad - b.dy.double()), ("dgamma", dg, g.grad),
                            ("dbeta", db, be.grad), ("dw", dw, w.grad)):
        err = (got.double() - want).norm() / want.norm()
        assert err <= 8 * u, f"{name}: {float(err):.2e}"


@pytest.mark.gpu
def test_branch_on_another_stream_and_in_graphs():
    """The same results on a side stream, and from two captured graphs replayed in turn after
    their inputs have changed."""
    a, b = Branch(300, 136, 264, "bf16", seed=1), Branch(70, 64, 72, "bf16", seed=2)
    want = [[t.clone() for t in k.forward_backward()] for k in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = a.forward_backward(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want[0]))
    graphs, outs = [], []
    for k in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(k.forward_backward())
        graphs.append(g)
    saved = a.x.clone()
    a.x.mul_(2)
    graphs[0].replay()
    assert not torch.equal(outs[0][0], want[0][0])
    a.x.copy_(saved)
    for _ in range(2):
        for g in graphs:
            g.replay()
    for o, wv in zip(outs, want):
        assert all(torch.equal(p, q) for p, q in zip(o, wv))
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(1, 72, 40), (7, 136, 72), (30, 264, 24), (300, 200, 136)], ids=lambda s: "x".join(map(str, s)))
def test_every_store_in_bounds(shape, dtype, monkeypatch):
    """The debug build checks every hand-indexed store against its buffer."""
    import os
    path = os.path.join(os.path.dirname(cb.library_path()), "libdgrad_debug.so")
    if not os.path.exists(path):
        pytest.skip("libdgrad_debug.so not built")
    monkeypatch.setattr(cb, "_LIB_PATH", path)
    monkeypatch.setattr(cb, "_lib", None)
    M, C, F = shape
    x, w, dh = _inputs(M, C, F, dtype, seed=M)
    h, z = cb.gated_forward(x, w, preact=True)
    dx, dw = cb.gated_backward(dh, x, z, w)
    cb.check_status()
    _check_forward(x, w, "silu", dtype, h, z, "debug")
    _check_backward(dh, x, z, w, "silu", dtype, dx, dw, "debug")
