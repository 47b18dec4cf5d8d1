"""Plain float64 references of the training operators.  Imported by tests only."""
from __future__ import annotations

import numpy as np

K1, K2 = np.uint32(0x9E3779B1), np.uint32(0x6A09E667)
BLOCK = 256


def mix(x):
    """The 32-bit mixing of the 8-bit moments' rounding."""
    x = np.asarray(x, dtype=np.uint32).copy()
    with np.errstate(over="ignore"):
        x ^= x >> np.uint32(16)
        x *= K1
        x ^= x >> np.uint32(15)
        x *= K2
        return x ^ (x >> np.uint32(16))


def uniform(seed, step, tensor, first, n):
    """The uniform numbers of elements [first, first + n) of a tensor; first even."""
    with np.errstate(over="ignore"):
        key = mix(mix(np.uint32(seed) ^ (np.uint32(step) * K1)) + np.uint32(tensor))
        pair = np.arange(first // 2, first // 2 + (n + 1) // 2, dtype=np.uint64)
        h = mix(pair.astype(np.uint32) ^ mix(key + (pair >> np.uint64(32)).astype(np.uint32)))
    u = np.stack([h & np.uint32(0xFFFF), h >> np.uint32(16)], 1).reshape(-1)[:n]
    return u.astype(np.float64) / 65536


def value_m(c, scale):
    c = c.astype(np.float64) / 127
    return np.repeat(scale.astype(np.float64), BLOCK)[:c.size] * c * np.abs(c)


def value_v(c, scale):
    return np.repeat(scale.astype(np.float64), BLOCK)[:c.size] * (c.astype(np.float64) / 255) ** 4


def place(x, power, levels):
    """Where the magnitudes x lie among the codes of their block, in codes: c plus
    the share of the way from c's value to the next one's; and the blocks' scales."""
    pad = -x.size % BLOCK
    b = np.pad(x, (0, pad)).reshape(-1, BLOCK)
    top = b.max(1)
    share = b / np.where(top > 0, top, 1)[:, None]
    c = np.clip(np.floor(share ** (1 / power) * levels), 0, levels)
    lo, hi = (c / levels) ** power, ((c + 1) / levels) ** power
    return (c + (share - lo) / (hi - lo)).reshape(-1)[:x.size], top


def adamw(w, g, m, v, t, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01):
    """One step in float64: w, m, v, and the update (lr times the quotient)."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g ** 2
    up = lr * (m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return w - lr * weight_decay * w - up, m, v, up
