"""CPU oracle for the AdamW step and the gradients' norm.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  The moments and the 8-bit codes are
defined by fp32 operations each rounded on its own, so they are formed here in numpy's fp32 and
have to be met bit for bit; weights and norms are formed in float64.
"""
from __future__ import annotations

import numpy as np

from oracle import branch

F = np.float32
BLOCK = 256


def moments(m, v, g, scale, beta1, beta2):
    """m', v' (fp32) from fp32 moments and fp32 gradients."""
    g = g * F(scale)
    return m * F(beta1) + g * F(1.0 - beta1), v * F(beta2) + (g * F(1.0 - beta2)) * g


def weights(w, m, v, step, lr, beta1, beta2, eps, wd):
    """(p', the update's part of it) in float64 from the new moments."""
    m, v = m.astype(np.float64), v.astype(np.float64)
    up = lr * (m / (1 - beta1 ** step)) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return w.astype(np.float64) * (1 - lr * wd) - up, up


def _value(c, power):
    q = c * c
    return q if power == 2 else q * q


def decode_m(c, top):
    f = c.astype(F)
    return ((f * np.abs(f)) * F(1 / 16129)) * np.repeat(top, BLOCK)[:c.size]


def decode_v(c, top):
    return (_value(c.astype(F), 4) * F(1 / 4228250625)) * np.repeat(top, BLOCK)[:c.size]


def encode(x, power, draws=None):
    """(codes, maxima) of fp32 x (n,): signed codes for power 2, unsigned for 4; draws: 16 bits each."""
    most = F(127 if power == 2 else 255)
    n = x.size
    pad = np.zeros(-(-n // BLOCK) * BLOCK, dtype=F)
    pad[:n] = x
    b = np.abs(pad).reshape(-1, BLOCK)
    top = b.max(axis=1)
    with np.errstate(all="ignore"):
        k = np.where(top < F(2.0 ** -60), F(2.0 ** 64), np.where(top > F(2.0 ** 60), F(2.0 ** -64), F(1)))
        inv = np.where(top > 0, (F(1) / (top * k)) * _value(most, power), F(0)).astype(F)
        w = ((b * k[:, None]) * inv[:, None]).reshape(-1)
        # low: the largest code whose value is at most w
        table = _value(np.arange(int(most) + 2).astype(F), power)
        low = np.searchsorted(table, w, side="right") - 1
        low = np.clip(low, 0, int(most))
        step = table[low + 1] - table[low]
        d = np.full(w.shape, F(32768)) if draws is None else draws.astype(F)
        up = (w - table[low]) * F(65536) > step * d
    c = np.minimum(low + up, int(most))
    c = c[:n]
    if power == 4:
        c = np.where((x > 0) & (c < 1), 1, c)
        return c.astype(np.uint8), top
    return np.where(x < 0, -c, c).astype(np.int8), top


def draws(first, n, seed, offset):
    """(for m, for v): 16 bits for each of n elements counted from `first` (a multiple of 256)."""
    b = np.arange(first // 4, first // 4 + -(-n // 4), dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    ctr = np.stack([b & low, b >> np.uint64(32), np.full_like(b, offset & 0xFFFFFFFF), np.full_like(b, offset >> 32)], axis=1)
    words = branch.philox(ctr, (seed & 0xFFFFFFFF, seed >> 32)).reshape(-1)[:n]
    return (words & np.uint64(0xFFFF)).astype(np.int64), (words >> np.uint64(16)).astype(np.int64)


def norm(arrays):
    return float(np.sqrt(sum(float((a.astype(np.float64) ** 2).sum()) for a in arrays)))
