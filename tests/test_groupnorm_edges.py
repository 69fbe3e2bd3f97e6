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
