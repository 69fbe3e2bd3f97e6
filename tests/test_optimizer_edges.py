"""The AdamW step, its states and the gradients' norm at their edges: subnormal eps; tensors that have no
memory, have shrunk or are not plain tensors; copies of states; autograd's knowledge of a step."""
import copy
import pickle
import subprocess
import sys

import numpy as np
import pytest

import convolution_backward_b200 as cb
import test_optimizer as to
from oracle import optim

torch = pytest.importorskip("torch")

HYPER = to.HYPER


def _described(ts):
    was = [cb._Array(np.zeros(len(ts), dtype=t)) for t in (np.uint64, np.int64, np.int64)]
    cb._lists().describe(ts, *(w.at for w in was))
    return [w.at for w in was], was


@pytest.mark.parametrize("change", ["narrow", "resize", "type", "order", "replace", "none", "reshape"])
def test_changed_tensors_are_seen(change):
    """At the same address, too (on the CPU: nothing here touches the elements)."""
    a, b = torch.zeros(7), torch.zeros(4, 4)
    at, was = _described([a, b])
    assert was[0].a.tolist() == [a.data_ptr(), b.data_ptr()] and was[1].a.tolist() == [7, 16]
    assert cb._lists().same([a, b], *at)
    where = b.data_ptr()
    if change == "narrow":
        b.data = b.data[:2]
    elif change == "resize":
        b.resize_(3, 3)
    elif change == "type":
        b.data = b.data.view(torch.int32)
    elif change == "order":
        b.data = b.data.t()
    elif change == "replace":
        b.data = b.data.clone()
    elif change == "reshape":
        b.data = b.data.view(2, 8)
    assert (b.data_ptr() == where) == (change != "replace")
    assert cb._lists().same([a, b], *at) == (change in ("none", "reshape"))


# Calls with something that is no plain tensor, in a process of their own: an exception that leaves native code ends it.
WRAPPED = """
import sys
import numpy as np
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.fx.experimental.symbolic_shapes import ShapeEnv
import convolution_backward_b200 as cb

L = cb._lists()
arrays = [cb._Array(np.zeros(4, dtype=t)) for t in (np.uint64, np.int64, np.int64)]
at = [a.at for a in arrays]
calls = {
    "norm": lambda x: cb.grad_norm([x]),
    "read": lambda x: L.read([x], None, "gradients", at[0], at[1]),
    "like": lambda x: L.read([x], [x], "gradients", at[0], 0),
    "describe": lambda x: L.describe([x], *at),
    "same": lambda x: L.same([x], *at),
}
env = ShapeEnv()


def run(f):
    if sys.argv[1] == "grad":
        torch.func.grad(lambda x: (f(x), x.sum())[1])(torch.empty(2, 3, device="cuda"))
    elif sys.argv[1] == "vmap":
        torch.vmap(lambda x: (f(x), x)[1])(torch.empty(2, 3, device="cuda"))
    else:
        f(torch.empty(env.create_unbacked_symint(), 3, device="cuda"))


with FakeTensorMode(shape_env=env):
    for name, f in calls.items():
        print("trying", name, file=sys.stderr, flush=True)
        try:
            run(f)
        except (RuntimeError, ValueError):
            print(name)
"""


@pytest.mark.parametrize("wrap", ["grad", "vmap", "symbolic"])
def test_wrapped_tensors_raise(wrap):
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", WRAPPED, wrap], capture_output=True, text=True,
                       cwd=to.os.path.dirname(to.os.path.dirname(to.os.path.abspath(__file__))), timeout=300)
    assert r.returncode == 0, r.stderr[:2000]
    assert r.stdout.split() == ["norm", "read", "like", "describe", "same"]


def test_tensors_without_memory_are_refused_on_the_host():
    """A fake tensor's address is its offset, as a released one's: 0 stands for no tensor in every table and argument."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        x, i = torch.empty(8, device="cuda"), torch.empty(1, dtype=torch.int64, device="cuda")
        at = [cb._Array(np.zeros(4, dtype=np.uint64)) for _ in range(3)]
        for t in (x, x[3:]):
            for like in (None, [t]):
                with pytest.raises(ValueError, match="storage"):
                    cb._lists().read([t], like, "gradients", at[0].at, at[1].at)
            with pytest.raises(ValueError, match="storage"):
                cb._lists().describe([t], *(a.at for a in at))
            with pytest.raises(ValueError, match="storage"):
                cb._ptr(t)
        with pytest.raises(ValueError, match="storage"):
            cb._scalar(x[:1], torch.float32, x.device, "lr")
        with pytest.raises(ValueError, match="storage"):
            cb._scalar(i, torch.int64, x.device, "step")
        with pytest.raises(ValueError, match="storage"):
            cb.adamw_state([x])
        with pytest.raises(ValueError, match="storage"):
            cb.grad_norm([x])
        assert cb._lists().read([x[:0]], None, "gradients", at[0].at, at[1].at) == (0, 0)
        assert cb._ptr(x[:0]) == 0 and cb._ptr(None) is None
    y = torch.zeros(10)
    assert cb._ptr(y[3:]) == y.data_ptr() + 12
    at, was = _described([y])
    y.untyped_storage().resize_(20)
    where = y.data_ptr()
    assert not cb._lists().same([y], *at), where


def test_copies_of_states_are_made_from_their_tensors():
    """A copied attribute would be the address of the first state's tables, which a step writes to."""
    s = object.__new__(cb.AdamWState)
    s.params, s.m, s.v, s.master, s.m_max, s.v_max = (torch.ones(3),), (torch.zeros(3),), (torch.zeros(3),), None, None, None
    s._grads = cb._Array(np.zeros(1, dtype=np.uint64))
    for again in (copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))):
        with pytest.raises(ValueError, match="CUDA"):      # the constructor sees them
            again(s)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_copied_states_step_on_their_own(bits):
    _, grads, state = to._make([700, 3, 0, 256], "bf16", "bf16", True, bits, seed=31)
    to._step(state, grads, 1)
    deep, pickled = copy.deepcopy(state), pickle.loads(pickle.dumps(state))
    shared = copy.copy(state)
    assert [t.data_ptr() for t in shared._all] == [t.data_ptr() for t in state._all]
    for other in (deep, pickled):
        ours = {t.data_ptr() for t in state._all if t.numel()}
        assert not ours & {t.data_ptr() for t in other._all}
        assert all(torch.equal(a, b) for a, b in zip(state._all, other._all))
    before = [t.clone() for t in state._all]
    to._step(deep, grads, 2)
    assert all(torch.equal(a, b) for a, b in zip(before, state._all))
    to._step(shared, grads, 2)
    assert all(torch.equal(a, b) for a, b in zip(deep._all, state._all))
    del state, shared
    to._step(pickled, grads, 2)
    assert all(torch.equal(a, b) for a, b in zip(deep._all, pickled._all))
    cb.check_status()


@pytest.mark.gpu
def test_released_tensors_are_refused():
    def gone(*shape, dtype=torch.float32, rows=None):
        """A tensor, or its rows from `rows` on, whose storage was released after it was made."""
        t = torch.ones(*shape, dtype=dtype, device="cuda")[rows:]
        t.untyped_storage().resize_(0)
        return t

    p, q = torch.ones(600, device="cuda"), torch.ones(5, device="cuda")
    for bits in (32, 8):
        state = cb.adamw_state([p, q], bits=bits)
        g, h = torch.ones(600, device="cuda"), torch.ones(5, device="cuda")
        before = [t.clone() for t in state._all]
        for bad in (gone(5), gone(9, rows=4)):
            with pytest.raises(ValueError, match="storage"):
                cb.adamw_step(state, [g, bad], 1, 1e-3)
            with pytest.raises(ValueError, match="storage"):
                cb.grad_norm([g, bad])
        for kw in ({"grad_scale": gone(1)}, {"lr": gone(1)}, {"step": gone(1, dtype=torch.int64)}):
            with pytest.raises(ValueError, match="storage"):
                cb.adamw_step(state, [g, h], **{"step": 1, "lr": 1e-3, **kw})
        assert all(torch.equal(a, b) for a, b in zip(before, state._all))
        with pytest.raises(ValueError, match="storage"):
            cb.adamw_state([gone(5)], bits=bits)
        state.m[1].untyped_storage().resize_(0)
        with pytest.raises(ValueError, match="storage"):
            cb.adamw_step(state, [g, h], 1, 1e-3)
    x, w = torch.ones(2, 3, 8, device="cuda"), torch.ones(8, device="cuda")
    for args in ((x, 2, gone(8), w), (x, 2, w, gone(8)), (gone(2, 3, 8), 2), (gone(3, 3, 8, rows=1), 2)):
        with pytest.raises(ValueError, match="storage"):
            cb.groupnorm_forward(*args)
    _, mean, rstd = cb.groupnorm_forward(x, 2, stats=True)
    for args in ((x, x, mean, rstd, gone(8)), (gone(3, 3, 8, rows=1), x, mean, rstd), (x, x, gone(2, 2), rstd)):
        with pytest.raises(ValueError, match="storage"):
            cb.groupnorm_backward(*args)
    with pytest.raises(ValueError, match="storage"):
        cb.layernorm_forward(x, gone(8))
    with pytest.raises(ValueError, match="storage"):
        cb.dropout_forward(x, 0.5, 1, residual=gone(2, 3, 8))
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_shrunk_tensors_are_refused(bits):
    """A parameter or state that is fewer elements at the same address: nothing runs on the old count."""
    for which in ("params", "m", "v"):
        p = torch.ones(600, device="cuda")
        state = cb.adamw_state([p, torch.ones(5, device="cuda")], bits=bits)
        keep = [t.clone() for t in state._all]
        whole = [t.data for t in state._all]
        t = getattr(state, which)[0]
        t.data = t.data[:4]
        g = torch.ones(4 if which == "params" else 600, device="cuda")
        with pytest.raises(ValueError, match="storage"):
            cb.adamw_step(state, [g, None], 1, 1e-3)
        with pytest.raises(ValueError, match="storage"):
            cb.adamw_step(state, [None, torch.ones(5, device="cuda")], 1, 1e-3)
        if bits == 8:
            out = [[torch.zeros(n, device="cuda") for n in (g.numel(), 5)] for _ in range(2)]
            with pytest.raises(ValueError, match="storage"):
                cb.adamw_moments(state, out=out)
        assert all(torch.equal(a, b) for a, b in zip(keep, whole))
        t.data = next(w for w in whole if w.data_ptr() == t.data_ptr())
        cb.adamw_step(state, [torch.ones(600, device="cuda"), None], 1, 1e-3)      # whole again
    cb.check_status()


def test_written_tensors_count_a_change():
    a, b, c, d = (torch.zeros(3) for _ in range(4))
    with torch.inference_mode():
        e = torch.zeros(3)
    at = np.array([1, 0], dtype=np.uint64)
    cb._lists().written([a, b, c, d, e], at.ctypes.data, 2)
    assert [t._version for t in (a, b, c, d)] == [1, 0, 1, 0]
    with pytest.raises(TypeError):
        cb._lists().written((a,), at.ctypes.data, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_a_graph_that_needs_the_old_weights_raises(bits):
    w, idle = (torch.ones(300, device="cuda", requires_grad=True) for _ in range(2))
    state = cb.adamw_state([w, idle], bits=bits)
    loss, other = (w * w).sum(), (idle * idle).sum()
    versions = [t._version for t in state.params]
    cb.adamw_step(state, [torch.ones(300, device="cuda"), None], 1, 1e-3)
    assert [t._version - v for t, v in zip(state.params, versions)] == [1, 0]
    half = cb.adamw_state([torch.ones(3, dtype=torch.bfloat16, device="cuda")], bits=bits, master=True)
    before = [t._version for t in (*half.params, *half.master)]
    cb.adamw_step(half, [torch.ones(3, dtype=torch.bfloat16, device="cuda")], 1, 1e-3)
    assert [t._version - v for t, v in zip((*half.params, *half.master), before)] == [1, 1]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    other.backward()
    assert torch.equal(idle.grad, 2 * torch.ones_like(idle))
    (w * w).sum().backward()
    assert torch.equal(w.grad, 2 * w.detach())
    if bits == 8:
        out = [[torch.zeros(300, device="cuda") for _ in range(2)] for _ in range(2)]
        cb.adamw_moments(state, out=out)
        assert all(t._version == 1 for ts in out for t in ts)
    with pytest.raises(cb.DgradError):
        cb.adamw_step(state, [w.grad, None], 0, 1e-3)
    assert w._version == versions[0] + 1         # refused: nothing was written
    with torch.inference_mode():
        cb.adamw_step(state, [w.grad, None], 2, 1e-3)
        p = torch.ones(5, device="cuda")
        cb.adamw_step(cb.adamw_state([p], bits=bits), [torch.ones(5, device="cuda")], 1, 1e-3)
    assert (p < 1).all()
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-40, 1.2e-38, 1e-30, 1e-13])
def test_small_eps(eps, bits):
    """Down to fp32's smallest numbers: where the moments are zero the update is 0/eps = 0 (at eps 0: NaN); where v' is
    zero and m' is not, m'/eps; elsewhere eps does not count.  Bounds: test_optimizer's weights."""
    n = 1000
    r = np.random.default_rng(4)
    h = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=float(np.float32(eps)), wd=0.1)
    w = r.normal(size=n).astype(np.float32)
    g = (1e-2 * r.normal(size=n)).astype(np.float32)
    g[::3] = 0
    g[1::3][:100] = 1e-30 * r.normal(size=100)          # whose square is zero
    g[256:512] = 0                                      # a block of nothing
    params = [torch.from_numpy(w).cuda()]
    state = cb.adamw_state(params, bits=bits)
    cb.adamw_step(state, [torch.from_numpy(g).cuda()], 1, h["lr"], (h["beta1"], h["beta2"]), eps, h["wd"])
    zero = np.zeros(n, dtype=np.float32)
    with np.errstate(all="ignore"):
        m, v = optim.moments(zero, zero, g, 1.0, h["beta1"], h["beta2"])
        ref, up = optim.weights(w.astype(np.float64), m, v, 1, **h)
    got = to._np(state.params[0]).astype(np.float64)
    nan = np.isnan(ref)
    assert nan.any() == (eps == 0) and (np.isnan(got) == nan).all()
    far = ~nan & (np.abs(ref) > 3.4e38)                 # m'/eps past fp32's range
    assert (np.isinf(got[far]) & (np.sign(got[far]) == np.sign(ref[far]))).all()
    near = ~nan & ~far
    bound = to.E32 * np.abs(ref) + 3 * to.E32 * np.abs(w) + 2.0 ** -20 * np.abs(up)
    assert (np.abs(got[near] - ref[near]) <= bound[near]).all()
    cb.check_status()
