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
        with np.errstate(over="ignore"):
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


def activation_errors(g, err_g, act: str):
    """Largest errors of (act(g), act'(g)) from fp32 steps and a g that is off by err_g.

    Curved range, |g| < 24: both forms have slopes of at most 1.13. The exponent's argument carries
    |g| 2^-24 twice, the exponential, the sum and the reciprocal 2^-23 or less each; so s (or
    (1 + tanh) / 2) is off by s (1 - s) (|g| + 1) 2^-23 + 1.5 s 2^-23, act by |g| times that and
    act' by at most 1 + |g| times it and the roundings of its products: 2^-20 (1 + |g|) max(1, |g|)
    and 2^-21 (1 + |g|) cover them (silu at g = 10: 20 2^-23 of 44; gelu's own factor,
    g / 2 (1 + 3 b g^2) c, is 9 where 1 - tanh^2 still differs from 0 in fp32, |g| <= 5.3).
    Outside it exp(-|g|) is below 2^-34: the sums round to their larger term, the reciprocal of 1
    is 1, and act is g or 0, act' 1 or 0, up to |g| exp(-|g|) < 2^-29 and four roundings."""
    A = np.abs(g)
    curved = A - err_g < 24.0
    flat = 1e-8                      # |g + 2| exp(-|g|) at 24 is 1e-9: the slopes left there
    slope_a = np.where(curved, 1.13, np.where(g < 0, flat, 1.13))
    err_a = slope_a * err_g + np.where(curved, 2.0 ** -20 * (1.0 + A) * np.maximum(1.0, A), 2.0 ** -22 * A)
    err_s = np.where(curved, 1.13, flat) * err_g + np.where(curved, 2.0 ** -21 * (1.0 + A), 2.0 ** -22)
    return err_a, err_s


def bounds(x, wg, wu, wd, act: str, half_step: float, dy=None, g_half_step: float | None = None):
    """Largest errors of y, or with dy of (dx, dWg, dWu, dWd).

    half_step: the storage type's largest relative rounding error (bf16 2^-8, fp32 2^-24).
    A sum of K fp32 products is off by at most K 2^-24 times the sum of their magnitudes; the
    activation and its derivative by activation_errors.
    """
    x, wg, wu, wd = (np.asarray(a, np.float64) for a in (x, wg, wu, wd))
    e, u32 = half_step, 2.0 ** -24
    (T, D), F = x.shape, wg.shape[0]
    A = np.abs
    g, u = x @ wg.T, x @ wu.T
    a, slope = activation(g, act)
    err_g, err_u = D * u32 * (A(x) @ A(wg).T), D * u32 * (A(x) @ A(wu).T)
    err_a, err_s = activation_errors(g, err_g, act)
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
