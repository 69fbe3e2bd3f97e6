"""Group norm where its statistics are hard to form: constant groups, means far above the spread,
infinities, sums at the end of fp32's range; and which of the two ways serves which size.

Tolerances (e = 2^-24, ulp: the distance of the fp32 neighbours of a value):
  constant groups   every difference to the mean is 0: equality.
  far means         x = base + j/64 with whole |j| <= 128 and base a multiple of 1/64 around 3000 are exact in fp32, and so
                    are their differences to any fp32 number near base.  A block's mean is rounded
                    once (half an ulp), the joined mean once more; what the sums of the differences lose,
                    (S + 160) e of 4 at most, is below a twentieth of an ulp of 3000 (2^-12) up to S = 50 and, as
                    they cancel around a centre, is taken as such at every size here: 1.1 ulp.
"""
import numpy as np
import pytest

import convolution_backward_b200 as cb
import test_branch_ops as tb
import test_groupnorm as tg
from oracle import branch

torch = pytest.importorskip("torch")

E32, TYPES, IDS = tg.E32, tg.TYPES, tg.IDS
to64, within = tb.to64, tb.within


@pytest.fixture(params=["auto", "s", "c"], ids=["auto", "streaming", "cluster"])
def way(request, monkeypatch):
    """The library's own choice (with what it keeps of it), the streaming way, the cluster way wherever it fits."""
    if request.param == "auto":
        monkeypatch.delenv("DGRAD_GN_WAY", raising=False)
    else:
        monkeypatch.setenv("DGRAD_GN_WAY", request.param)
    cb._gn_workspace.cache_clear()
    yield request.param
    cb._gn_workspace.cache_clear()


SHAPES = [(333, 21, 7), (256, 768, 32), (400, 64, 8), (4000, 24, 1), (50, 2056, 8), (1, 40, 2), (700, 100, 25)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_constant_groups_leave_beta(shape, dtype, way):
    """Values that sums round: the mean of equal values is the value, and the result beta."""
    S, C, G = shape
    t = TYPES[dtype][0]
    _, g, b, _ = tg._inputs(1, 1, C, dtype, seed=2)
    for v in (0.3, 100.1, -255.3, 3e4 / 7):
        row = (v * (1 + torch.arange(G, dtype=torch.float64) / 7)).to(t).cuda()
        x = row.repeat_interleave(C // G).expand(3, S, C).contiguous()
        y, mean, rstd = cb.groupnorm_forward(x, G, g, b, eps=1e-5, stats=True)
        assert torch.equal(mean, row.float().expand(3, G)), v
        assert torch.equal(y, b.expand_as(y)), v
        one = torch.tensor(1e-5).rsqrt().item()
        assert ((rstd / one - 1).abs() <= 4 * E32).all(), v
    y = cb.groupnorm_forward(x, G, g, b, eps=0.0)
    assert torch.isnan(y).all()                # 0 times an infinite rstd
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_means_far_above_the_spread(shape, way):
    S, C, G = shape
    r = np.random.default_rng(S + C)
    N = 3
    base = 3000.25 + r.integers(-4000, 4000, size=(N, 1, G, 1)) / 64
    X = (base + r.integers(-128, 129, size=(N, S, G, C // G)) / 64).reshape(N, S, C)
    x = torch.from_numpy(X.astype(np.float32)).cuda()
    assert np.array_equal(to64(x), X)
    _, mean, rstd = cb.groupnorm_forward(x, G, eps=1e-5, stats=True)
    _, rm, rr = branch.groupnorm(X, G, np.ones(C), np.zeros(C), 1e-5)
    within(mean, rm, 1.1 * np.spacing(rm.astype(np.float32)).astype(np.float64), "mean")
    A = 1 + np.square((X - branch._spread(rm, C)) * branch._spread(rr, C)).max()
    within(rstd, rr, rr * (A * (S + 136) / 2 + 4) * E32 + 0.5 * rr ** 3 * np.spacing(3100.0, dtype=np.float32) ** 2, "rstd")
    cb.check_status()



@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("far", [6, 30, 100, 1000])
@pytest.mark.parametrize("shape", [(333, 21, 7), (256, 768, 32), (4000, 24, 1)], ids=IDS)
def test_means_on_both_sides_of_the_bound(shape, far, dtype, way):
    """From some spreads to many, under test_groupnorm's bounds."""
    S, C, G = shape
    x, g, b, dy = tg._inputs(2, S, C, dtype, seed=far, offset=0.0)
    x = (x.float() + far).to(x.dtype)
    y, mean, rstd = cb.groupnorm_forward(x, G, g, b, act="silu", stats=True)
    tg._check_fwd(x, G, g, b, 1e-5, "silu", dtype, y, mean, rstd, "forward", whole=False)
    got = cb.groupnorm_backward(dy, x, mean, rstd, g, b, act="silu")
    tg._check_bwd(dy, x, g, b, mean, rstd, "silu", dtype, got, "backward")
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[2] > 1 and s[0] > 1], ids=IDS)
def test_a_far_mean_changes_its_own_group_alone(shape, way):
    S, C, G = shape
    D = C // G
    x, g, b, dy = tg._inputs(3, S, C, "f32", seed=S)
    y, mean, rstd = cb.groupnorm_forward(x, G, g, b, act="silu", stats=True)
    z = x.clone()
    z[1, :, D:2 * D] += 3000.0
    z[2, :, C - D:] = 100.1
    hit = torch.zeros(3, G, dtype=torch.bool, device="cuda")
    hit[1, 1] = hit[2, G - 1] = True
    y2, mean2, rstd2 = cb.groupnorm_forward(z, G, g, b, act="silu", stats=True)
    assert torch.equal(mean2[~hit], mean[~hit]) and torch.equal(rstd2[~hit], rstd[~hit])
    wide = hit.repeat_interleave(D, dim=1)[:, None, :].expand_as(y)
    assert torch.equal(y2[~wide], y[~wide]) and (mean2[2, G - 1] == np.float32(100.1)).item()
    got = cb.groupnorm_backward(dy, z, mean2, rstd2, g, b, act="silu")
    tg._check_bwd(dy, z, g, b, mean2, rstd2, "silu", "f32", got, "backward")
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(333, 21, 7), (400, 64, 8), (4000, 24, 1), (20000, 16, 4), (7, 40, 5)], ids=IDS)
def test_an_infinity_makes_its_groups_statistics_nan(shape, way):
    """At the first position, a middle one (in another block) and the last."""
    S, C, G = shape
    D = C // G
    x, g, b, _ = tg._inputs(3, S, C, "f32", seed=21)
    y0, mean0, rstd0 = cb.groupnorm_forward(x, G, g, b, stats=True)
    for bad in (float("inf"), float("-inf"), float("nan")):
        for n, s in ((0, 0), (1, S // 2), (2, S - 1)):
            z = x.clone()
            z[n, s, C - 1] = bad
            y, mean, rstd = cb.groupnorm_forward(z, G, g, b, stats=True)
            hit = torch.zeros(3, G, dtype=torch.bool, device="cuda")
            hit[n, G - 1] = True
            assert torch.isnan(mean[hit]).all() and torch.isnan(rstd[hit]).all(), (bad, s)
            assert torch.equal(mean[~hit], mean0[~hit]) and torch.equal(rstd[~hit], rstd0[~hit]), (bad, s)
            assert torch.isnan(y[n, :, C - D:]).all()
            y[n, :, C - D:] = y0[n, :, C - D:]
            assert torch.equal(y, y0)
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(333, 21, 7), (400, 64, 8), (4000, 24, 1), (7, 40, 5)], ids=IDS)
def test_sums_up_to_the_range(shape, way):
    """m max|x| just inside fp32's range: the means are numbers, rstd is 0 and beta is left.  Past it a group's
    results are its own formula's or NaN, never another number."""
    S, C, G = shape
    D, m = C // G, S * (C // G)
    r = np.random.default_rng(5)
    _, g, b, _ = tg._inputs(1, 1, C, "f32", seed=3)
    X = (r.uniform(0.2, 1.0, size=(2, S, C)) * (3.3e38 / m)).astype(np.float32)
    x = torch.from_numpy(X).cuda()
    y, mean, rstd = cb.groupnorm_forward(x, G, g, b, stats=True)
    _, rm, _ = branch.groupnorm(X.astype(np.float64), G, np.ones(C), np.zeros(C), 0.0)
    within(mean, rm, (S + 132) * E32 * rm, "mean")
    assert not rstd.any() and torch.equal(y, b.expand_as(y))
    y, mean, rstd = cb.groupnorm_forward(x * m, G, g, b, stats=True)
    rm *= m
    ok = torch.isnan(mean) | ((mean.double() - torch.from_numpy(rm).cuda()).abs() <= 1e-3 * torch.from_numpy(rm).cuda())
    assert ok.all() and (torch.isnan(rstd) == torch.isnan(mean)).all() and not torch.nan_to_num(rstd).any()
    nan = torch.isnan(mean).repeat_interleave(D, dim=1)[:, None, :].expand_as(y)
    assert torch.isnan(y[nan]).all() and torch.equal(y[~nan], b.expand_as(y)[~nan])
    cb.check_status()


@pytest.mark.gpu
def test_far_means_captured_and_on_two_streams(way):
    """Replays on inputs with and without far means, and two calls at once."""
    N, S, C, G = 4, 200, 96, 8
    near, g, b, _ = tg._inputs(N, S, C, "f32", seed=41)
    far = near + 3000.0
    far[1] = 100.1
    want = [cb.groupnorm_forward(t, G, g, b, act="silu", stats=True) for t in (near, far)]
    x = near.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cb.groupnorm_forward(x, G, g, b, act="silu", stats=True)
    for k in (1, 0, 1, 1, 0):
        x.copy_((near, far)[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want[k]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for t, s in zip((near, far), streams):
            with torch.cuda.stream(s):
                got.append(cb.groupnorm_forward(t, G, g, b, act="silu", stats=True))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for w, o in zip(want, got) for p, q in zip(w, o))
    z = far.clone()
    assert cb.groupnorm_forward(z, G, g, b, act="silu", out=z) is z and torch.equal(z, want[1][0])     # in place
    cb.check_status()


# ------------------------------------------------------------------ which way, and sizes at the ends

def _ways(N, S, C, G, dtype):
    """(forward, backward): "cluster" or "streaming", from the workspaces: the cluster way needs none forward, and
    2 C sums for each of its N K blocks along the positions (K up to 8) backward."""
    cb._gn_workspace.cache_clear()
    t = TYPES[dtype][0]
    fwd = cb.groupnorm_forward_workspace_bytes(N, S, C, G, t)
    bwd = cb.groupnorm_backward_workspace_bytes(N, S, C, G, t)
    clusters = [-(-(N * k * 2 * C * 4) // 16) * 16 for k in (1, 2, 4, 8)]
    return "streaming" if fwd else "cluster", "cluster" if bwd in clusters else "streaming"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("cluster", [1, 2, 4, 8])
@pytest.mark.parametrize("shape", [(3, 100, 96, 8, 2), (2, 150, 40, 1, 1), (1, 300, 66, 6, 4), (5, 9, 256, 32, 5), (2, 130, 24, 8, 3)], ids=IDS)
def test_every_cluster_size_runs(shape, cluster, dtype, monkeypatch):
    """Sizes whose slices fit the shared memory of every cluster: the way that was named is the one that runs."""
    N, S, C, G, slices = shape
    monkeypatch.setenv("DGRAD_GN_WAY", "c")
    monkeypatch.setenv("DGRAD_GN_CLUSTER", str(cluster))
    monkeypatch.setenv("DGRAD_GN_SLICES", str(slices))
    assert _ways(N, S, C, G, dtype) == ("cluster", "cluster")
    assert cb.groupnorm_backward_workspace_bytes(N, S, C, G, TYPES[dtype][0]) == -(-(N * cluster * 2 * C * 4) // 16) * 16
    x, g, b, dy = tg._inputs(N, S, C, dtype, seed=S + cluster)
    y, mean, rstd = cb.groupnorm_forward(x, G, g, b, act="silu", stats=True)
    tg._check_fwd(x, G, g, b, 1e-5, "silu", dtype, y, mean, rstd, "forward")
    got = cb.groupnorm_backward(dy, x, mean, rstd, g, b, act="silu")
    tg._check_bwd(dy, x, g, b, mean, rstd, "silu", dtype, got, "backward")
    x[0, :, :C // G] = 100.1
    y, mean, rstd = cb.groupnorm_forward(x, G, g, b, stats=True)
    assert torch.equal(y[0, :, :C // G], b[:C // G].expand(S, C // G))
    tg._check_fwd(x, G, g, b, 1e-5, None, dtype, y, mean, rstd, "one constant group")
    cb.check_status()
    cb._gn_workspace.cache_clear()


def test_the_choice_takes_both_ways(monkeypatch):
    monkeypatch.delenv("DGRAD_GN_WAY", raising=False)
    assert _ways(2, 64, 512, 32, "bf16") == ("cluster", "cluster")
    assert _ways(16, 4096, 384, 32, "bf16") == ("streaming", "streaming")
    monkeypatch.setenv("DGRAD_GN_WAY", "s")
    assert _ways(2, 64, 512, 32, "bf16") == ("streaming", "streaming")
    monkeypatch.setenv("DGRAD_GN_WAY", "c")
    assert _ways(16, 1024, 384, 32, "bf16") == ("cluster", "cluster")
    assert _ways(1, 1 << 20, 8, 1, "bf16") == ("streaming", "streaming")      # fits nowhere
    cb._gn_workspace.cache_clear()


@pytest.mark.gpu
def test_kept_choices_of_many_sizes(monkeypatch):
    """More sizes in turn than a thread keeps choices for, forward and backward, twice over."""
    monkeypatch.delenv("DGRAD_GN_WAY", raising=False)
    cb._gn_workspace.cache_clear()
    sizes = [(2, 64, 512, 32), (1, 16384, 8, 2), (3, 33, 21, 7), (4, 256, 96, 32), (2, 64, 512, 16), (2, 65, 512, 32), (1, 5000, 64, 8),
             (7, 1, 40, 5), (2, 512, 64, 32), (64, 2, 512, 32), (5, 700, 66, 6), (1, 64, 512, 32)]
    ins = [tg._inputs(N, S, C, "f32", seed=k) for k, (N, S, C, G) in enumerate(sizes)]
    first = None
    for turn in range(2):
        outs = []
        for (N, S, C, G), (x, g, b, dy) in zip(sizes, ins):
            y, mean, rstd = cb.groupnorm_forward(x, G, g, b, act="silu", stats=True)
            outs.append((y, mean, rstd, *cb.groupnorm_backward(dy, x, mean, rstd, g, b, act="silu")))
            if turn == 0:
                tg._check_fwd(x, G, g, b, 1e-5, "silu", "f32", y, mean, rstd, f"{N}x{S}x{C}")
                tg._check_bwd(dy, x, g, b, mean, rstd, "silu", "f32", outs[-1][3:], f"{N}x{S}x{C}")
        first = first or outs
    assert all(torch.equal(p, q) for a, b in zip(first, outs) for p, q in zip(a, b))
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(8192, 1, 64, 8), (3000, 3, 40, 5), (70000, 1, 8, 2), (513, 5, 33, 3), (2, 3, 65536, 32), (1, 2, 65535, 5)],
                         ids=IDS)
def test_many_samples_and_the_most_channels(shape, dtype, way):
    N, S, C, G = shape
    x, g, b, dy = tg._inputs(N, S, C, dtype, seed=C + S)
    y, mean, rstd = cb.groupnorm_forward(x, G, g, b, act="silu", stats=True)
    tg._check_fwd(x, G, g, b, 1e-5, "silu", dtype, y, mean, rstd, "forward")
    got = cb.groupnorm_backward(dy, x, mean, rstd, g, b, act="silu")
    tg._check_bwd(dy, x, g, b, mean, rstd, "silu", dtype, got, "backward")
    cb.check_status()


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 99])
def test_gradients_past_32_bits(C):
    """More than 2^31 elements, all different samples: small whole numbers with mean 0 and rstd 1, so that n = x and every
    sum is a whole number that fp32 holds (of random signs: far below 2^24).  dgamma and dbeta are those numbers rounded to
    bf16; dX carries the divisions by m and four operations, and its rounding."""
    N, S, G = 34, -(-(1 << 31) // (33 * C)), 3
    D, m = C // G, S * (C // G)
    r = torch.Generator(device="cuda").manual_seed(2)
    xi, di = (torch.randint(-2, 3, (N, S, C), dtype=torch.int8, device="cuda", generator=r) for _ in range(2))
    assert xi.numel() > 1 << 31
    x, dy = xi.bfloat16(), di.bfloat16()
    g = (1 + torch.arange(C, device="cuda") % 2).bfloat16()
    mean, rstd = torch.zeros(N, G, device="cuda"), torch.ones(N, G, device="cuda")
    dx, dg, db = cb.groupnorm_backward(dy, x, mean, rstd, g)
    want_g, want_b = torch.zeros(C, dtype=torch.int64, device="cuda"), torch.zeros(C, dtype=torch.int64, device="cuda")
    for n in range(N):
        a, d = xi[n].double(), di[n].double()
        want_g += (a * d).sum(0).long()
        want_b += d.sum(0).long()
        q = d * g.double()
        qa = q.view(S, G, D).sum((0, 2)) / m
        qb = (q * a).view(S, G, D).sum((0, 2)) / m
        ref = q - qa.repeat_interleave(D) - a * qb.repeat_interleave(D)
        bound = 2.0 ** -8 * ref.abs() + 1.01 * 4 * E32 * (q.abs() + qa.abs().repeat_interleave(D) + 2 * (a * qb.repeat_interleave(D)).abs())
        assert ((dx[n].double() - ref).abs() <= bound + 1e-30).all(), n
    assert torch.equal(dg, want_g.float().bfloat16()) and torch.equal(db, want_b.float().bfloat16())
    assert want_g.abs().max() < 1 << 24 and want_b.abs().max() < 1 << 24
    cb.check_status()
