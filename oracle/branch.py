"""fp64 CPU oracle for the residual branch's operators: layer norm, group norm, the gated
pointwise block and dropout, each with its gradients.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Plain numpy in float64 from
the definitions; nothing here is shared with the CUDA path.  tests/test_branch_ops.py
pins the gradients against central differences and the generator against published
values.
"""
from __future__ import annotations

import math

import numpy as np


def layernorm(x, gamma, beta, eps):
    """(y, mean, rstd) over the last axis of x (M, C)."""
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    return (x - mean[:, None]) * rstd[:, None] * gamma + beta, mean, rstd


def layernorm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta) with the given statistics."""
    n = (x - mean[:, None]) * rstd[:, None]
    q = dy * gamma
    dx = rstd[:, None] * (q - q.mean(axis=1)[:, None] - n * (q * n).mean(axis=1)[:, None])
    return dx, (dy * n).sum(axis=0), dy.sum(axis=0)


def _erf(v):
    return np.vectorize(math.erf, otypes=[np.float64])(v)


def act(name, g):
    """(act(g), act'(g))."""
    if name in ("silu", "sigmoid"):
        s = np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))
        return (g * s, s * (1 + g * (1 - s))) if name == "silu" else (s, s * (1 - s))
    if name == "relu":
        return np.maximum(g, 0.0), (g > 0).astype(np.float64)
    if name == "gelu":
        cdf = 0.5 * (1 + _erf(g / math.sqrt(2)))
        return g * cdf, cdf + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    assert name == "gelu_tanh"
    k = math.sqrt(2 / math.pi)
    t = np.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def _spread(stat, C):
    """(N, G) statistics to (N, 1, C)."""
    return np.repeat(stat, C // stat.shape[1], axis=1)[:, None, :]


def groupnorm(x, G, gamma, beta, eps, name=None):
    """(y, mean, rstd) of x (N, S, C) in G groups of channels; name: an activation or None."""
    N, S, C = x.shape
    g = x.reshape(N, S, G, C // G)
    mean = g.mean(axis=(1, 3))
    rstd = 1.0 / np.sqrt(((g - mean[:, None, :, None]) ** 2).mean(axis=(1, 3)) + eps)
    z = (x - _spread(mean, C)) * _spread(rstd, C) * gamma + beta
    return (z if name is None else act(name, z)[0]), mean, rstd


def groupnorm_backward(dy, x, gamma, beta, mean, rstd, name=None, slope=None):
    """(dx, dgamma, dbeta) with the given statistics; slope: act'(z) where it is known already."""
    N, S, C = x.shape
    G = mean.shape[1]
    n = (x - _spread(mean, C)) * _spread(rstd, C)
    if slope is None:
        slope = np.ones_like(n) if name is None else act(name, n * gamma + beta)[1]
    dz = dy * slope
    q = (dz * gamma).reshape(N, S, G, C // G)
    ng = n.reshape(N, S, G, C // G)
    a, b = q.mean(axis=(1, 3)), (q * ng).mean(axis=(1, 3))
    dx = _spread(rstd, C) * (dz * gamma - _spread(a, C) - n * _spread(b, C))
    return dx, (dz * n).sum(axis=(0, 1)), dz.sum(axis=(0, 1))


def gated(x, w, name):
    """(h, z): z = x w^T = [g | u], h = act(g)*u; w (2F, C)."""
    z = x @ w.T
    F = w.shape[0] // 2
    return act(name, z[:, :F])[0] * z[:, F:], z


def gated_dz(dh, z, name):
    """[dg | du]: the gradient at the pre-activations."""
    F = z.shape[1] // 2
    a, d = act(name, z[:, :F])
    return np.concatenate([dh * z[:, F:] * d, dh * a], axis=1)


def gated_backward(dh, x, z, w, name):
    """(dx, dw) with the given pre-activations."""
    dz = gated_dz(dh, z, name)
    return dz @ w, dz.T @ x


def philox(counter, key):
    """Philox-4x32-10: counter (n, 4) and key (2,), 32-bit words -> (n, 4)."""
    c = [np.asarray(counter)[:, i].astype(np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> sh) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=1)


def dropout_keep(n, p, seed, offset):
    """(keep (n,) of truth values, scale)."""
    b = np.arange((n + 7) // 8, dtype=np.uint64)
    ctr = np.stack([b & np.uint64(0xFFFFFFFF), b >> np.uint64(32), np.full_like(b, offset & 0xFFFFFFFF),
                    np.full_like(b, offset >> 32)], axis=1)
    words = philox(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    draws = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], axis=2).reshape(-1)[:n]
    t = int(round(p * 65536))
    return draws >= t, 65536.0 / (65536 - t) if t < 65536 else 0.0
