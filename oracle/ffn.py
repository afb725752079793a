"""Gated feed-forward block in NumPy float64, forward and backward, from its formulas:

    g = x Wg^T, u = x Wu^T, h = act(g) u, y = h Wd^T
    dh = dy Wd, du = dh act(g), dg = dh u act'(g)
    dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T h

``bounds`` gives, for each result, how far fp32 arithmetic with the intermediates h, dg and
du rounded to a storage type may be from it, element by element.
"""

from __future__ import annotations

import numpy as np


def activation(g, act: str):
    """(act(g), act'(g))."""
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu_tanh":
        c, b = np.sqrt(2.0 / np.pi), 0.044715
        t = np.tanh(c * (g + b * g ** 3))
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * b * g * g)
    raise ValueError(act)


def forward(x, wg, wu, wd, act: str):
    x, wg, wu, wd = (np.asarray(a, np.float64) for a in (x, wg, wu, wd))
    a, _ = activation(x @ wg.T, act)
    return (a * (x @ wu.T)) @ wd.T


def backward(dy, x, wg, wu, wd, act: str):
    """(dx, dWg, dWu, dWd)."""
    dy, x, wg, wu, wd = (np.asarray(a, np.float64) for a in (dy, x, wg, wu, wd))
    g, u = x @ wg.T, x @ wu.T
    a, slope = activation(g, act)
    dh = dy @ wd
    dg, du = dh * u * slope, dh * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ (a * u)


def bounds(x, wg, wu, wd, act: str, half_step: float, dy=None, g_half_step: float | None = None):
    """Largest errors of y, or with dy of (dx, dWg, dWu, dWd).

    half_step: the storage type's largest relative rounding error (bf16 2^-8, fp32 2^-24).
    A sum of K fp32 products is off by at most K 2^-24 times the sum of their magnitudes. The
    activation and its derivative have slopes of at most 1.13 (both forms); evaluated in fp32
    they are off by at most 2^-20 (1 + |g|) relative to max(1, |g|) (the exponent's argument
    carries |g| 2^-24 log2 e, the exponential, the reciprocal and the products a few 2^-24).
    """
    x, wg, wu, wd = (np.asarray(a, np.float64) for a in (x, wg, wu, wd))
    e, u32 = half_step, 2.0 ** -24
    (T, D), F = x.shape, wg.shape[0]
    A = np.abs
    g, u = x @ wg.T, x @ wu.T
    a, slope = activation(g, act)
    err_g, err_u = D * u32 * (A(x) @ A(wg).T), D * u32 * (A(x) @ A(wu).T)
    own = 2.0 ** -20 * (1.0 + A(g)) * np.maximum(1.0, A(g))
    err_a, err_s = 1.13 * err_g + own, 1.13 * err_g + own
    h = a * u
    err_h = A(u) * err_a + A(a) * err_u + err_a * err_u + (e + 2 * u32) * A(h)
    more = 1.05  # products of two errors
    if dy is None:
        y = h @ wd.T
        return more * (err_h @ A(wd).T + F * u32 * (A(h) @ A(wd).T) + e * A(y))
    dy = np.asarray(dy, np.float64)
    eg = e if g_half_step is None else g_half_step
    dh = dy @ wd
    err_dh = D * u32 * (A(dy) @ A(wd))
    dg, du = dh * u * slope, dh * a
    err_du = A(a) * err_dh + A(dh) * err_a + (e + 2 * u32) * A(du)
    err_dg = A(u * slope) * err_dh + A(dh) * (A(slope) * err_u + A(u) * err_s) + (e + 4 * u32) * A(dg)
    dx = dg @ wg + du @ wu
    out = [err_dg @ A(wg) + err_du @ A(wu) + 2 * F * u32 * (A(dg) @ A(wg) + A(du) @ A(wu)) + e * A(dx)]
    for d, err, other in ((dg, err_dg, x), (du, err_du, x)):
        out.append(err.T @ A(other) + T * u32 * (A(d).T @ A(other)) + eg * A(d.T @ other))
    out.append(A(dy).T @ err_h + T * u32 * (A(dy).T @ A(h)) + eg * A(dy.T @ h))
    return tuple(more * o for o in out)
