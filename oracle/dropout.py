"""Dropout from a counter (the formulas of ``muon_drop`` in ``include/muon.h``) in plain integers:
Philox4x32-10 after Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3" (SC
2011), sections 3.3 and 5."""

from __future__ import annotations

import math

import numpy as np

M32 = 0xFFFFFFFF


def philox(counter, key, rounds=10):
    """Four 32-bit words from a 4-word counter and a 2-word key."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & M32, (a >> 32) ^ c[3] ^ k[1], a & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def numbers(n, seed, offset):
    """The 16-bit numbers of elements 0 .. n - 1."""
    out = np.empty(n, np.int64)
    split = lambda x: (x & M32, (x >> 32) & M32)  # noqa: E731
    for b in range((n + 7) // 8):
        words = philox((*split(b), *split(offset)), split(seed))
        for e in range(min(8, n - 8 * b)):
            out[8 * b + e] = (words[e // 2] >> (16 * (e % 2))) & 0xFFFF
    return out


def threshold(p):
    """p in 32 bits, as the library takes it."""
    return math.floor(float(np.float32(p)) * 65536.0 + 0.5)


def dropout(x, p, seed, offset, residual=None):
    x = np.asarray(x, np.float64)
    c = threshold(p)
    keep = (numbers(x.size, seed, offset) >= c).reshape(x.shape)
    out = np.where(keep, np.where(keep, x, 0.0) * (65536.0 / (65536 - c) if c < 65536 else 0.0), 0.0)
    return out if residual is None else out + np.asarray(residual, np.float64)
