"""The AdamW step over many tensors (32-bit and 8-bit states), what 8-bit states stand for, and the
gradients' norm, against oracle/optim.py, and their refusals.

Moments and codes are defined by fp32 operations and have to be met bit for bit.  Tolerances of the
rest (u: the type's half step relative to the value, eta half its smallest subnormal; e = 2^-24):
  weights  the decayed weight carries 2 roundings; the update's root and reciprocal are approximate
           (2^-22 each), with 6 roundings more: 2^-20 of it; their sum one more.
  norm     formed in 64 bits, rounded once: e, and e more for the division by it.
"""
import ctypes
import os

import numpy as np
import pytest

import convolution_backward_b200 as cb
import test_branch_ops as tb
from oracle import branch, optim

torch = pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, 1, 2, 3
FAKE = tb.FAKE
E32 = 2.0 ** -24
TYPES = tb.TYPES
to64, within = tb.to64, tb.within
DEBUG_LIB = os.path.join(os.path.dirname(cb.library_path()), "libdgrad_debug.so")


class _Tensor(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("param", "grad", "m", "v", "master", "m_max", "v_max")] + [("n", ctypes.c_int64)]


def _opt(**kw):
    h = cb._AdamW()
    h.lr, h.beta1, h.beta2, h.eps, h.weight_decay, h.step, h.state_bits = 1e-3, 0.9, 0.999, 1e-8, 0.1, 1, 32
    for k, v in kw.items():
        setattr(h, k, v)
    return h


def _tensor(i=0, **kw):
    t = _Tensor()
    for k, name in enumerate(("param", "grad", "m", "v", "master", "m_max", "v_max")):
        setattr(t, name, FAKE * (1 + k) + i * 0x100000 if name in ("param", "grad", "m", "v") else None)
    t.n = 100
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _list(*ts):
    return (_Tensor * len(ts))(*ts)


# ------------------------------------------------------------------- the oracle

def test_oracle_codes():
    r = np.random.default_rng(0)
    x = (r.normal(size=1000) * np.exp(3 * r.normal(size=1000))).astype(np.float32)
    x[:256] = 0
    for power, most in ((2, 127), (4, 255)):
        v = x if power == 2 else np.abs(x)
        c, top = optim.encode(v, power)
        got = (optim.decode_m if power == 2 else optim.decode_v)(c, top).astype(np.float64)
        unit = np.repeat(top.astype(np.float64), 256)[:1000]
        share = np.where(unit > 0, np.abs(v) / np.where(unit > 0, unit, 1), 0)
        low = np.floor(share ** (1 / power) * most)
        half = (((low + 1) / most) ** power - (low / most) ** power) / 2 * unit
        least = np.where((power == 4) & (v > 0), unit / most ** 4, 0)      # a v above zero keeps a code
        assert (np.abs(got - v) <= half * (1 + 1e-5) + least).all()
        assert (c[:256] == 0).all() and np.abs(c).max() == most
    # random draws: the mean of many codes' values is the value
    v = np.zeros(256, dtype=np.float32)
    v[0], v[1:] = 1.0, 0.3217
    tries = [optim.decode_v(*optim.encode(v, 4, draws=r.integers(0, 65536, size=256)))[1:] for _ in range(200)]
    step = np.diff(np.unique(np.concatenate(tries)))
    # 51000 draws between two neighbours: their mean is within six deviations
    assert len(step) == 1 and abs(np.mean(tries) - 0.3217) < 6 * 0.5 * step[0] / np.sqrt(51000)


# ------------------------------------------------------------------ host checks

def test_step_refusals():
    step = cb.lib().dgrad_adamw_step

    def call(t=None, pt=0, gt=0, count=None, opt=None, **kw):
        t = _list(_tensor()) if t is None else t
        return step(len(t) if count is None else count, t, pt, gt, ctypes.byref(_opt(**kw)) if opt is None else opt, None)

    nan, inf = float("nan"), float("inf")
    assert step(1, _list(_tensor()), 0, 0, None, None) == INVALID
    for bad in ({"count": -1}, {"pt": 3}, {"gt": -1}, {"state_bits": 16}, {"beta1": 1.0}, {"beta1": -0.1}, {"beta2": 1.0},
                {"beta2": nan}, {"eps": -1e-9}, {"eps": nan}, {"eps": inf}, {"lr": nan}, {"lr": inf}, {"weight_decay": nan},
                {"step": 0}, {"step": -1}, {"stochastic": 1}, {"stochastic": 2, "state_bits": 8}, {"state_bits": 8}):
        assert call(**bad) == INVALID, bad
    assert step(1, None, 0, 0, ctypes.byref(_opt()), None) == INVALID
    for bad in ({"param": None}, {"m": None}, {"v": None}, {"n": -1}):
        assert call(_list(_tensor(**bad))) == INVALID, bad
    assert call(_list(_tensor(), _tensor(1, master=9 * FAKE)), pt=1, gt=1) == INVALID       # a master copy for one
    assert call(_list(_tensor(master=9 * FAKE))) == UNSUPPORTED
    assert call(pt=0, gt=1) == UNSUPPORTED
    assert call(pt=1, gt=2) == UNSUPPORTED
    assert call(_list(_tensor(n=1 << 41))) == UNSUPPORTED
    for bad in ({"param": FAKE + 2}, {"grad": FAKE + 1}, {"m": FAKE + 2}, {"v": FAKE + 1}):
        assert call(_list(_tensor(**bad))) == ALIGNMENT, bad
    assert call(_list(_tensor(param=FAKE + 1)), pt=1, gt=1) == ALIGNMENT
    assert call(_list(_tensor(master=FAKE + 2)), pt=1, gt=1) == ALIGNMENT
    assert call(_list(_tensor(m_max=FAKE + 2, v_max=FAKE)), state_bits=8) == ALIGNMENT
    for k in ("lr_device", "grad_scale"):
        assert call(**{k: FAKE + 2}) == ALIGNMENT
    assert call(step_device=FAKE + 4) == ALIGNMENT
    assert call(count=0) == OK


def test_check_finds_shared_memory():
    check = cb.lib().dgrad_adamw_check
    assert check(2, _list(_tensor(), _tensor(1)), 0, 0, 32) == OK
    assert check(2, _list(_tensor(), _tensor()), 0, 0, 32) == INVALID                      # the same tensor twice
    assert check(1, _list(_tensor(m=FAKE)), 0, 0, 32) == INVALID
    assert check(1, _list(_tensor(v=3 * FAKE + 396)), 0, 0, 32) == INVALID
    assert check(1, _list(_tensor(v=3 * FAKE + 400)), 0, 0, 32) == OK
    assert check(1, _list(_tensor(grad=FAKE)), 0, 0, 32) == INVALID
    assert check(2, _list(_tensor(), _tensor(1, grad=2 * FAKE)), 0, 0, 32) == OK            # gradients are read only
    assert check(1, _list(_tensor(m_max=9 * FAKE, v_max=9 * FAKE)), 0, 0, 8) == INVALID
    assert check(1, _list(_tensor(m_max=9 * FAKE, v_max=9 * FAKE + 4)), 0, 0, 8) == OK
    assert check(1, _list(_tensor(n=0, m=FAKE)), 0, 0, 32) == OK
    assert check(0, None, 0, 0, 32) == OK


def test_moments_and_norm_refusals():
    L = cb.lib()
    ptrs = (ctypes.c_void_p * 1)(FAKE)
    out2 = (ctypes.c_void_p * 1)(2 * FAKE)
    t = _list(_tensor(m_max=9 * FAKE, v_max=10 * FAKE))
    assert L.dgrad_adamw_moments(-1, t, ptrs, out2, None) == INVALID
    assert L.dgrad_adamw_moments(1, None, ptrs, out2, None) == INVALID
    assert L.dgrad_adamw_moments(1, t, None, out2, None) == INVALID
    assert L.dgrad_adamw_moments(1, _list(_tensor()), ptrs, out2, None) == INVALID           # no maxima
    assert L.dgrad_adamw_moments(1, t, (ctypes.c_void_p * 1)(FAKE + 2), out2, None) == ALIGNMENT
    assert L.dgrad_adamw_moments(0, None, None, None, None) == OK
    nb = ctypes.c_size_t()
    assert L.dgrad_grad_norm_workspace(5, None) == INVALID
    assert L.dgrad_grad_norm_workspace(-1, ctypes.byref(nb)) == INVALID
    assert L.dgrad_grad_norm_workspace(0, ctypes.byref(nb)) == OK and nb.value == 0
    assert L.dgrad_grad_norm_workspace(5, ctypes.byref(nb)) == OK and nb.value > 0

    def norm(count=1, g=FAKE, n=100, dtype=1, limit=1.0, out=3 * FAKE, ws=4 * FAKE, size=nb.value):
        return L.dgrad_grad_norm(count, (ctypes.c_void_p * 1)(g), (ctypes.c_int64 * 1)(n), dtype, limit, out, ws, size, None)

    for bad in ({"count": -1}, {"g": None}, {"n": -1}, {"dtype": 3}, {"limit": -1.0}, {"limit": float("nan")}, {"out": None},
                {"ws": None}, {"size": nb.value - 1}, {"out": FAKE}, {"out": FAKE + 196}, {"ws": FAKE + 16},
                {"out": 4 * FAKE + 8}):
        assert norm(**bad) == INVALID, bad
    for bad in ({"g": FAKE + 1}, {"out": 3 * FAKE + 2}, {"ws": 4 * FAKE + 8}):
        assert norm(**bad) == ALIGNMENT, bad
    assert norm(n=1 << 41) == UNSUPPORTED


def test_binding_refusals():
    with pytest.raises(ValueError, match="CUDA"):
        cb.grad_norm([torch.zeros(4)])
    with pytest.raises(ValueError, match="at least one"):
        cb.grad_norm([])
    with pytest.raises(ValueError, match="CUDA"):
        cb.adamw_state([torch.zeros(4)])
    with pytest.raises(ValueError, match="at least one"):
        cb.adamw_state([])
    with pytest.raises(ValueError, match="bits"):
        cb.adamw_state([torch.zeros(4)], bits=16)


@pytest.mark.gpu
def test_state_and_step_refusals():
    mk = lambda n, t=torch.float32: torch.zeros(n, dtype=t, device="cuda")
    p, m, v = mk(10), mk(10), mk(10)
    with pytest.raises(ValueError, match="share"):
        cb.AdamWState([p, p], [m, mk(10)], [v, mk(10)])
    with pytest.raises(ValueError, match="share"):
        cb.AdamWState([p], [m], [m])
    with pytest.raises(ValueError, match="m: expected 1"):
        cb.AdamWState([p], [], [v])
    with pytest.raises(ValueError, match="v must have shape"):
        cb.AdamWState([p], [m], [mk(11)])
    with pytest.raises(TypeError, match="m must be"):
        cb.AdamWState([p], [mk(10, torch.float16)], [v])
    with pytest.raises(ValueError, match="m_max"):
        cb.AdamWState([p], [mk(10, torch.int8)], [mk(10, torch.uint8)])
    with pytest.raises(ValueError, match="m_max and v_max"):
        cb.AdamWState([p], [m], [v], m_max=[mk(1)], v_max=[mk(1)])
    with pytest.raises(ValueError, match="v_max must have shape"):
        cb.AdamWState([p], [mk(10, torch.int8)], [mk(10, torch.uint8)], m_max=[mk(1)], v_max=[mk(2)])
    with pytest.raises(cb.DgradError):
        cb.AdamWState([p], [m], [v], master=[mk(10)])        # fp32 parameters are their own
    with pytest.raises(ValueError, match="contiguous"):
        cb.AdamWState([mk(20)[::2]], [m], [v])
    s = cb.AdamWState([p], [m], [v])
    g = mk(10)
    step = lambda gs, **kw: cb.adamw_step(s, gs, kw.pop("step", 1), kw.pop("lr", 1e-3), **kw)
    with pytest.raises(ValueError, match="1 gradients"):
        step([g, g])
    with pytest.raises(ValueError, match="shapes"):
        step([mk(11)])
    with pytest.raises(ValueError, match="shapes"):
        step([g.view(2, 5)])
    with pytest.raises(TypeError, match="float32"):
        step([mk(10, torch.bfloat16)])
    with pytest.raises(ValueError, match="contiguous"):
        step([mk(20)[::2]])
    with pytest.raises(ValueError, match="share"):
        step([p])
    with pytest.raises(ValueError, match="CUDA"):
        step([torch.zeros(10)])
    with pytest.raises(ValueError, match="seed"):
        step([g], seed=1)
    with pytest.raises(TypeError, match="grad_scale"):
        step([g], grad_scale=mk(1, torch.float64))
    with pytest.raises(ValueError, match="lr must have one"):
        step([g], lr=mk(2))
    with pytest.raises(TypeError, match="step must be"):
        step([g], step=mk(1, torch.int32))
    for bad in ({"step": 0}, {"lr": float("nan")}, {"betas": (1.0, 0.9)}, {"eps": -1.0}):
        with pytest.raises(cb.DgradError):
            step([g], **bad)
    assert not p.any() and not m.any()
    p.data = mk(10)
    with pytest.raises(ValueError, match="storage"):
        step([g])
    with pytest.raises(ValueError, match="32-bit"):
        cb.adamw_moments(s, out=([g], [mk(10)]))
    s8 = cb.adamw_state([mk(10)], bits=8)
    with pytest.raises(ValueError, match="share"):
        cb.adamw_moments(s8, out=([g], [g]))
    with pytest.raises(ValueError, match="shapes"):
        cb.adamw_moments(s8, out=([g], [mk(9)]))
    with pytest.raises(TypeError):
        cb.grad_norm([g, mk(3, torch.float16)])
    with pytest.raises(ValueError, match="contiguous"):
        cb.grad_norm([mk(20)[::2]])


# ------------------------------------------------------------------ the step

HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, wd=0.1)
SIZES = [1, 3, 4, 255, 256, 257, 2048, 2049, 5000, 7, 100_001]


def _make(sizes, dtype, gdtype, master, bits, seed, misalign=0):
    r = np.random.default_rng(seed)

    def mk(a, t):
        """A tensor whose first element lies `misalign` elements behind an aligned one."""
        a = torch.from_numpy(np.asarray(a, dtype=np.float32)).to(t)
        buf = torch.zeros(a.numel() + misalign, dtype=t, device="cuda")
        buf[misalign:].copy_(a)
        return buf[misalign:]

    t = TYPES[dtype][0]
    unlike = [np.exp(2 * r.normal()) for _ in sizes]
    params = [mk(r.normal(size=n) * 0.1, t) for n in sizes]
    grads = [mk(r.normal(size=n) * 1e-2 * k * np.exp(r.normal(size=n)), TYPES[gdtype][0]) for n, k in zip(sizes, unlike)]
    more = {"master": [mk(to64(p) + 1e-4 * r.normal(size=n), torch.float32) for p, n in zip(params, sizes)]} if master else {}
    m = [(r.normal(size=n) * 3e-3 * k).astype(np.float32) for n, k in zip(sizes, unlike)]
    v = [((r.normal(size=n) * 1e-2 * k) ** 2).astype(np.float32) for n, k in zip(sizes, unlike)]
    if bits == 32:
        return params, grads, cb.AdamWState(params, [mk(a, torch.float32) for a in m], [mk(a, torch.float32) for a in v], **more)

    def codes(a, power, t):
        c, top = optim.encode(a, power)
        buf = torch.zeros(c.size + misalign, dtype=t, device="cuda")
        buf[misalign:].copy_(torch.from_numpy(c))
        return buf[misalign:], torch.from_numpy(top).cuda()

    cm, cv = [codes(a, 2, torch.int8) for a in m], [codes(a, 4, torch.uint8) for a in v]
    return params, grads, cb.AdamWState(params, [c for c, _ in cm], [c for c, _ in cv], m_max=[x for _, x in cm],
                                        v_max=[x for _, x in cv], **more)


def _np(t):
    return t.detach().cpu().numpy().reshape(-1)


def _snapshot(state):
    lists = (state.params, state.m, state.v, state.master, state.m_max, state.v_max)
    return [None if ts is None else [t.clone() for t in ts] for ts in lists]


def _check_step(before, state, grads, dtype, what, step=1, scale=1.0, seed=None, offset=0, lr=None, untouched=()):
    """The state after one step against the oracle's from the snapshot before it."""
    _, u, eta = TYPES[dtype]
    h = dict(HYPER, lr=HYPER["lr"] if lr is None else lr)
    P, M, V, W, MM, VM = before
    first = 0
    for i, g in enumerate(grads):
        n = P[i].numel()
        blocks = -(-n // 256) * 256
        if g is None or i in untouched:
            for old, new in ((P, state.params), (M, state.m), (V, state.v), (W, state.master), (MM, state.m_max), (VM, state.v_max)):
                assert old is None or torch.equal(old[i], new[i]), f"{what} tensor {i} was left out"
            first += blocks
            continue
        G = _np(g.float())
        if state.bits == 32:
            m, v = _np(M[i]), _np(V[i])
        else:
            m, v = optim.decode_m(_np(M[i]), _np(MM[i])), optim.decode_v(_np(V[i]), _np(VM[i]))
        m, v = optim.moments(m, v, G, scale, h["beta1"], h["beta2"])
        if state.bits == 32:
            assert np.array_equal(_np(state.m[i]), m, equal_nan=True), f"{what} m of tensor {i}"
            assert np.array_equal(_np(state.v[i]), v, equal_nan=True), f"{what} v of tensor {i}"
        else:
            dm = dv = None
            if seed is not None:
                pad = lambda d: np.concatenate([d, np.zeros(blocks - n, dtype=d.dtype)])
                dm, dv = (pad(d) for d in optim.draws(first, n, seed, offset))
            for got, top, x, power, d in ((state.m[i], state.m_max[i], m, 2, dm), (state.v[i], state.v_max[i], v, 4, dv)):
                c, t = optim.encode(x, power, d)
                assert np.array_equal(_np(top), t), f"{what} maxima of tensor {i}"
                bad = np.flatnonzero(_np(got) != c)
                assert bad.size == 0, f"{what} codes of tensor {i}: {bad.size} off, first {bad[0]}: {_np(got)[bad[0]]} {c[bad[0]]}"
        w0 = to64(W[i] if W is not None else P[i]).reshape(-1)
        ref, up = optim.weights(w0, m, v, step, **h)
        err = 3 * E32 * np.abs(w0) + 2.0 ** -20 * np.abs(up)
        if W is not None:
            within(state.master[i].view(-1), ref, E32 * np.abs(ref) + err, f"{what} master {i}")
            assert torch.equal(state.params[i], state.master[i].to(state.params[i].dtype)), f"{what} copy {i}"
        else:
            within(state.params[i].view(-1), ref, u * np.abs(ref) + (1 + u) * err + eta, f"{what} param {i}")
        first += blocks


def _step(state, grads, step=1, **kw):
    cb.adamw_step(state, grads, step, kw.pop("lr", HYPER["lr"]), (HYPER["beta1"], HYPER["beta2"]), HYPER["eps"], HYPER["wd"], **kw)


COMBOS = [("f32", "f32", False), ("bf16", "bf16", False), ("bf16", "bf16", True), ("f16", "f16", True), ("f16", "f16", False),
          ("bf16", "f32", True), ("bf16", "f32", False), ("f16", "f32", True), ("f16", "f32", False)]


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["32", "8", "8s"])
@pytest.mark.parametrize("combo", COMBOS, ids=lambda c: f"{c[0]}-{c[1]}{'-master' if c[2] else ''}")
def test_steps(combo, mode):
    """Two steps, on aligned tensors and on ones an element off."""
    dtype, gdtype, master = combo
    for misalign in (0, 1):
        _, grads, state = _make(SIZES, dtype, gdtype, master, 32 if mode == "32" else 8, seed=3 + misalign, misalign=misalign)
        scale = torch.tensor([0.375], device="cuda")
        for k in (1, 2):
            seeds = dict(seed=0x123456789ABCDEF0 + k, offset=(k << 40) + 7) if mode == "8s" else {}
            before = _snapshot(state)
            _step(state, grads, k, grad_scale=scale, **seeds)
            _check_step(before, state, grads, dtype, f"step {k} off by {misalign}", k, 0.375, **seeds)
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_from_zero_states_and_left_out_tensors(bits):
    params = [torch.randn(n, device="cuda") for n in (300, 0, 5, 1000)]
    grads = [torch.randn_like(p) for p in params]
    state = cb.adamw_state(params, bits=bits)
    grads[2] = None
    for k in (1, 2, 3):
        before = _snapshot(state)
        _step(state, grads, k)
        _check_step(before, state, grads, "f32", f"step {k}", k)
    before = _snapshot(state)
    _step(state, [None] * 4, 4)
    _check_step(before, state, [None] * 4, "f32", "nothing")
    zero = [torch.zeros_like(p) for p in params]
    state = cb.adamw_state(params, bits=bits)
    before = _snapshot(state)
    _step(state, zero, 1)       # 0/(0 + eps): the decay alone
    _check_step(before, state, zero, "f32", "zeros")
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_a_scale_that_is_no_number_leaves_the_step_out(bits):
    _, grads, state = _make([500, 3], "bf16", "bf16", True, bits, seed=5)
    before = _snapshot(state)
    for s in (float("nan"), float("inf"), float("-inf")):
        _step(state, grads, 1, grad_scale=torch.tensor(s, device="cuda"))
    _check_step(before, state, [None, None], "bf16", "left out")
    grads[0][7] = float("inf")
    norm, scale = cb.grad_norm(grads, 1.0)
    assert torch.isinf(norm) and torch.isnan(scale)
    _step(state, grads, 1, grad_scale=scale)
    _check_step(before, state, [None, None], "bf16", "an infinite gradient")
    grads[0][7] = 1.0
    norm, scale = cb.grad_norm(grads, 1e-3)
    _step(state, grads, 1, grad_scale=scale)
    _check_step(before, state, grads, "bf16", "clipped", 1, scale.item())


@pytest.mark.gpu
def test_infinities_and_nan_stay_where_they_are():
    """32 bits: in their element; 8 bits: in the states of their 256, and in their own weight."""
    for bits in (32, 8):
        _, grads, state = _make([1000], "f32", "f32", False, bits, seed=6)
        grads[0][300], grads[0][900] = float("inf"), float("nan")
        clean = [g.clone() for g in grads]
        clean[0][300] = clean[0][900] = 0.5
        _, _, other = _make([1000], "f32", "f32", False, bits, seed=6)
        _step(state, grads)
        _step(other, clean)
        same = torch.ones(1000, dtype=torch.bool, device="cuda")
        same[[300, 900]] = False
        assert torch.equal(state.params[0][same], other.params[0][same])
        assert torch.isnan(state.params[0][[300, 900]]).all()
        m, v = cb.adamw_moments(state)
        if bits == 8:
            spoilt = torch.zeros(1000, dtype=torch.bool, device="cuda")
            spoilt[256:512] = spoilt[768:] = True
            assert torch.isnan(m[0][spoilt]).all() and torch.isnan(v[0][spoilt]).all()
            assert torch.isfinite(m[0][~spoilt]).all() and torch.isfinite(v[0][~spoilt]).all()
        else:
            assert torch.isfinite(m[0][same]).all() and torch.isfinite(v[0][same]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["8", "8s"])
@pytest.mark.parametrize("k", [-60, -35, -18, 15, 50])
def test_codes_over_the_range(k, mode):
    """Gradients of 2^k and their squares, down to where squares are subnormal or zero and up to where
    they pass fp32's range."""
    r = np.random.default_rng(100 + k)
    n = 256 * 20 + 11
    scale = 2.0 ** k * np.exp(2 * r.normal(size=(n // 256 + 1, 1)))
    g = (scale * r.normal(size=(n // 256 + 1, 256)) * np.exp(2 * r.normal(size=(n // 256 + 1, 256)))).reshape(-1)[:n]
    if k > 0:
        g = np.clip(g, -1.8e19, 1.8e19)
    g[5:200:7] = 0
    params, grads = [torch.zeros(n, device="cuda")], [torch.from_numpy(g.astype(np.float32)).cuda()]
    state = cb.adamw_state(params, bits=8)
    for step in (1, 2):
        seeds = dict(seed=11, offset=step) if mode == "8s" else {}
        before = _snapshot(state)
        _step(state, grads, step, **seeds)
        P, M, V, _, MM, VM = before
        with np.errstate(all="ignore"):
            m, v = optim.moments(optim.decode_m(_np(M[0]), _np(MM[0])), optim.decode_v(_np(V[0]), _np(VM[0])), _np(grads[0]), 1.0,
                                 HYPER["beta1"], HYPER["beta2"])
        blocks = -(-n // 256) * 256
        dm = dv = None
        if seeds:
            dm, dv = (np.concatenate([d, np.zeros(blocks - n, dtype=d.dtype)]) for d in optim.draws(0, n, 11, step))
        for got, top, x, power, d in ((state.m[0], state.m_max[0], m, 2, dm), (state.v[0], state.v_max[0], v, 4, dv)):
            c, t = optim.encode(x, power, d)
            assert np.array_equal(_np(top), t)
            assert np.array_equal(_np(got), c)
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_table_holds(bits):
    r = np.random.default_rng(1)
    sizes = [int(n) for n in np.exp(r.uniform(0, 9, size=1000))]
    _, grads, state = _make(sizes, "bf16", "bf16", True, bits, seed=8)
    grads[400] = grads[999] = None
    seeds = dict(seed=5, offset=9) if bits == 8 else {}
    before = _snapshot(state)
    _step(state, grads, 3, **seeds)
    _check_step(before, state, grads, "bf16", "1000 tensors", 3, **seeds)
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_device_step_and_rate_in_a_graph(bits):
    """A captured step reads its count, rate and scale in every replay."""
    _, grads, state = _make([700, 9000], "bf16", "bf16", True, bits, seed=9)
    start = _snapshot(state)
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    rate, scale = torch.zeros((), device="cuda"), torch.ones((), device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            count += 1
            _step(state, grads, count, lr=rate, grad_scale=scale)
    for ts, olds in zip((state.params, state.m, state.v, state.master, state.m_max, state.v_max), start):
        if ts is not None:
            for t, o in zip(ts, olds):
                t.copy_(o)
    torch.cuda.synchronize()
    for k, lr, s in ((1, 1e-2, 1.0), (2, 5e-3, 0.5), (3, 1e-3, 2.0)):
        rate.fill_(lr)
        scale.fill_(s)
        before = _snapshot(state)
        graph.replay()
        torch.cuda.synchronize()
        assert count.item() == k
        # the rate and 1 - rate decay are fp32 here
        _check_step(before, state, grads, "bf16", f"replay {k}", k, s, lr=float(np.float32(lr)))
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_device_scalars_that_say_nothing_leave_the_step_out(bits):
    _, grads, state = _make([700, 3], "f32", "f32", False, bits, seed=9)
    before = _snapshot(state)
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    _step(state, grads, zero)
    _step(state, grads, zero - 5)
    for bad in (float("nan"), float("inf")):
        _step(state, grads, 1, lr=torch.tensor(bad, device="cuda"))
    _check_step(before, state, [None, None], "f32", "left out")
    _step(state, grads, zero + 1)
    _check_step(before, state, grads, "f32", "step 1")


@pytest.mark.gpu
def test_replaced_states_and_shared_scalars_are_refused():
    _, grads, state = _make([300, 3], "f32", "f32", False, 8, seed=9)
    with pytest.raises(ValueError, match="must not share"):
        _step(state, grads, 1, grad_scale=state.params[0][:1])
    with pytest.raises(ValueError, match="must not share"):
        _step(state, grads, 1, lr=state.m_max[0][1:2])
    assert isinstance(state.params, tuple) and isinstance(state.m_max, tuple)
    state.m[1].data = state.m[1].clone()
    with pytest.raises(ValueError, match="storage"):
        _step(state, grads, 1)
    with pytest.raises(ValueError, match="storage"):
        cb.adamw_moments(state)


@pytest.mark.gpu
def test_one_tensor_past_32_bits():
    """More than 2^31 elements in one tensor, and one behind it in the list: its end against the same
    values alone."""
    n, tail = (1 << 31) + 1000, 5000
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    r = torch.Generator(device="cuda").manual_seed(3)
    p[-tail:] = torch.randn(tail, device="cuda", generator=r).bfloat16()
    g[-tail:] = torch.randn(tail, device="cuda", generator=r).bfloat16()
    at = (n - tail) // 256 * 256
    small_p, small_g = p[at:].clone(), g[at:].clone()
    state, small = cb.adamw_state([p, small_p], bits=8), cb.adamw_state([small_p.clone()], bits=8)
    _step(state, [g, small_g], 1)
    _step(small, [small_g], 1)
    assert torch.equal(state.params[0][at:], small.params[0]) and torch.equal(state.params[1], small.params[0])
    assert torch.equal(state.m[0][at:], small.m[0]) and torch.equal(state.v[0][at:], small.v[0])
    assert torch.equal(state.v_max[0][at // 256:], small.v_max[0]) and not state.m[0][:at].any()
    _step(state, [g, small_g], 2, seed=7, offset=1)
    first = -(-n // 256) * 256       # the second tensor's elements are counted from there
    before = optim.decode_m(_np(small.m[0]), _np(small.m_max[0]))
    m, _ = optim.moments(before, before, _np(small_g.float()), 1.0, HYPER["beta1"], HYPER["beta2"])
    d, _ = optim.draws(first, -(-m.size // 256) * 256, 7, 1)
    assert np.array_equal(_np(state.m[1]), optim.encode(m, 2, d)[0])
    ref = optim.norm([to64(g[-tail:])])
    assert abs(cb.grad_norm([g]).item() - ref) <= 2 * E32 * ref
    cb.check_status()


@pytest.mark.gpu
def test_on_another_stream():
    _, grads, state = _make([70_000, 33], "f32", "f32", False, 8, seed=10)
    before = _snapshot(state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm, scale = cb.grad_norm(grads, 1.0, stream=side)
    _step(state, grads, 1, grad_scale=scale, stream=side)
    m, v = cb.adamw_moments(state, stream=side)
    side.synchronize()
    _check_step(before, state, grads, "f32", "side stream", 1, scale.item())
    assert np.array_equal(_np(m[0]), optim.decode_m(_np(state.m[0]), _np(state.m_max[0])))


@pytest.mark.gpu
@pytest.mark.parametrize("misalign", [0, 1])
def test_moments(misalign):
    _, _, state = _make([1, 255, 256, 257, 70_001, 0], "f32", "f32", False, 8, seed=11, misalign=misalign)
    out = tuple([torch.full((p.numel() + 1,), 7.0, device="cuda")[misalign:p.numel() + misalign] for p in state.params] for _ in range(2))
    m, v = cb.adamw_moments(state)
    got = cb.adamw_moments(state, out=out)
    assert got[0][0] is out[0][0]
    for i in range(len(state)):
        assert np.array_equal(_np(m[i]), optim.decode_m(_np(state.m[i]), _np(state.m_max[i])))
        assert np.array_equal(_np(v[i]), optim.decode_v(_np(state.v[i]), _np(state.v_max[i])))
        assert torch.equal(m[i], out[0][i]) and torch.equal(v[i], out[1][i])
    s32 = cb.adamw_state([torch.zeros(5, device="cuda")])
    assert cb.adamw_moments(s32)[0] is s32.m
    cb.check_status()


# ------------------------------------------------------------------ the norm

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
def test_norm(dtype):
    r = np.random.default_rng(4)
    t = TYPES[dtype][0]
    for sizes in ([1], [5, 0, 4096, 4097, 100_003], [3] * 70, [int(n) for n in np.exp(r.uniform(0, 8, size=1700))], [3_000_017]):
        gs = []
        for k, n in enumerate(sizes):
            buf = torch.from_numpy(r.normal(size=n + 1).astype(np.float32)).to(t).cuda()
            gs.append(buf[k % 2:n + k % 2])         # every other one off the 16-byte grid
        ref = optim.norm([to64(g) for g in gs])
        norm, scale = cb.grad_norm(gs, 0.5)
        assert abs(norm.item() - ref) <= E32 * ref * 1.01
        want = min(1.0, 0.5 / (ref + 1e-6))
        assert abs(scale.item() - want) <= 4 * E32 * want
        again = cb.grad_norm(gs)
        assert torch.equal(again, norm)
    assert cb.grad_norm([torch.zeros(0, dtype=t, device="cuda")]).item() == 0
    assert cb.grad_norm([torch.zeros(9, dtype=t, device="cuda")], 1.0)[1].item() == 1
    cb.check_status()


@pytest.mark.gpu
def test_norm_over_the_range():
    big = torch.full((1000,), 3e38, device="cuda")
    assert torch.isinf(cb.grad_norm([big]))                      # beyond fp32 as a norm
    one = torch.full((1000,), 1e30, device="cuda")               # its squares alone are beyond it
    assert abs(cb.grad_norm([one]).item() / (1e30 * 1000 ** 0.5) - 1) < 1e-6
    small = torch.full((1000,), 1e-30, device="cuda")
    assert abs(cb.grad_norm([small]).item() / (1e-30 * 1000 ** 0.5) - 1) < 1e-6
    for bad in (float("nan"), float("inf")):
        one[777] = bad
        norm, scale = cb.grad_norm([small, one], 1.0)
        assert not torch.isfinite(norm) and torch.isnan(scale)


@pytest.mark.gpu
def test_norm_workspace_in_two_graphs():
    gs = [torch.randn(n, device="cuda") for n in (10, 50_000, 777)]
    ws = torch.full((cb.grad_norm_workspace_bytes(3),), 0xFF, dtype=torch.uint8, device="cuda")
    want = cb.grad_norm(gs, 1.0)
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(cb.grad_norm(gs, 1.0, workspace=ws))
        graphs.append(graph)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["32", "8s"])
def test_every_store_in_bounds(mode, monkeypatch):
    """Under the debug build, whose stores check their place."""
    if not os.path.exists(DEBUG_LIB):
        pytest.skip("libdgrad_debug.so not built")
    monkeypatch.setattr(cb, "_LIB_PATH", DEBUG_LIB)
    monkeypatch.setattr(cb, "_lib", None)
    for misalign in (0, 1):
        _, grads, state = _make(SIZES, "bf16", "f32", True, int(mode[0] + mode[1:].strip("s")), seed=2, misalign=misalign)
        seeds = dict(seed=3, offset=4) if mode == "8s" else {}
        before = _snapshot(state)
        norm, scale = cb.grad_norm(grads, 1.0)
        _step(state, grads, 5, grad_scale=scale, **seeds)
        _check_step(before, state, grads, "bf16", "debug", 5, scale.item(), **seeds)
        cb.adamw_moments(state)
    cb.check_status()


# ------------------------------------------------------------------ together

@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_a_convolution_block_trains_one_step(bits):
    """x -> group norm + silu -> 1x1 convolution, backward, the gradients' norm and a clipped step: every call
    against the oracle on the inputs that it was given."""
    N, H, W, C, K, G = 3, 9, 11, 64, 40, 8
    r = np.random.default_rng(21)
    mk = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()
    x, w = mk(r.normal(size=(N, H, W, C))), mk(r.normal(size=(K, C)) / 8)
    gamma, beta, dout = mk(1 + 0.2 * r.normal(size=C)), mk(0.2 * r.normal(size=C)), mk(r.normal(size=(N, H, W, K)))
    params = [w, gamma, beta]
    state = cb.adamw_state(params, bits=bits, master=True)
    for step in (1, 2):
        y, mean, rstd = cb.groupnorm_forward(x, G, gamma, beta, act="silu", stats=True)
        dy = cb.pointwise(dout, w)
        dw = (dout.view(-1, K).float().T @ y.view(-1, C).float()).to(torch.bfloat16)
        dx, dgamma, dbeta = cb.groupnorm_backward(dy, x, mean, rstd, gamma, beta, act="silu")
        grads = [dw, dgamma, dbeta]
        norm, scale = cb.grad_norm(grads, 1.0)
        before = _snapshot(state)
        X = to64(x).reshape(N, H * W, C)
        ref = branch.groupnorm_backward(to64(dy).reshape(N, H * W, C), X, to64(gamma), to64(beta), to64(mean), to64(rstd), "silu")
        for got, want in zip((dx.view(N, H * W, C), dgamma, dbeta), ref):
            assert np.linalg.norm(to64(got) - want) <= 2.0 ** -8 * np.linalg.norm(want)
        assert abs(norm.item() - optim.norm([to64(g) for g in grads])) <= 2 * E32 * norm.item()
        seeds = dict(seed=77, offset=step) if bits == 8 else {}
        _step(state, grads, step, grad_scale=scale, **seeds)
        _check_step(before, state, grads, "bf16", f"step {step}", step, scale.item(), **seeds)
    cb.check_status()
