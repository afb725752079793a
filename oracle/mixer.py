"""Linear attention with a decay for each head in float64, token by token (the formulas of
``muon_mix`` in ``include/muon.h``), its gradients by the reversed recurrence, and error bounds.

Arrays: q batch x tokens x heads x dim, k batch x tokens x kv_heads x dim, v batch x tokens x kv_heads x
dim_v, state batch x heads x dim x dim_v.
"""

from __future__ import annotations

import numpy as np


def _wide(x, heads):
    return np.repeat(np.asarray(x, np.float64), heads // x.shape[2], axis=2)


def _gamma(log_decay):
    with np.errstate(divide="ignore"):
        return np.exp(np.asarray(log_decay, np.float64))[:, None, None]


def _lengths(lengths, batch, tokens):
    if lengths is None:
        return np.full(batch, tokens)
    return np.clip(np.asarray(lengths), 0, tokens)


def forward(q, k, v, log_decay, scale, state=None, lengths=None):
    """(o, last states)."""
    q = np.asarray(q, np.float64)
    B, T, H, D = q.shape
    k, v, g = _wide(k, H), _wide(v, H), _gamma(log_decay)
    n = _lengths(lengths, B, T)
    last = np.zeros((B, H, D, v.shape[3])) if state is None else np.array(state, np.float64)
    o = np.zeros((B, T, H, v.shape[3]))
    for b in range(B):
        S = last[b]
        for t in range(n[b]):
            S = g * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            o[b, t] = scale * np.matmul(q[b, t][:, None, :], S)[:, 0]
        last[b] = S
    return o, last


def backward(do, q, k, v, log_decay, scale, state=None, lengths=None, d_final=None):
    """(dq, dk, dv, dstate)."""
    q, do = np.asarray(q, np.float64), np.asarray(do, np.float64)
    B, T, H, D = q.shape
    kv, E = k.shape[2], v.shape[3]
    k, v, g = _wide(k, H), _wide(v, H), _gamma(log_decay)
    n = _lengths(lengths, B, T)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    ds = np.zeros((B, H, D, E)) if d_final is None else np.array(d_final, np.float64)
    for b in range(B):
        S = np.zeros((H, D, E)) if state is None else np.asarray(state[b], np.float64)
        for t in range(n[b]):
            S = g * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            dq[b, t] = scale * np.matmul(S, do[b, t][:, :, None])[:, :, 0]
        dS = ds[b]
        for t in range(n[b] - 1, -1, -1):
            dS = dS + scale * q[b, t][:, :, None] * do[b, t][:, None, :]
            dk[b, t] = np.matmul(dS, v[b, t][:, :, None])[:, :, 0]
            dv[b, t] = np.matmul(k[b, t][:, None, :], dS)[:, 0]
            dS = g * dS
        ds[b] = dS
    shared = lambda x: x.reshape(B, T, kv, H // kv, -1).sum(3)  # noqa: E731
    return dq, shared(dk), shared(dv), ds


def sums32(tokens, dim, group=1):
    """Relative error of the kernels' fp32 arithmetic against the sum of a result's absolute terms.
    In steps of 2^-24: a dot product of up to 256 and one of 64 terms, one scaling of the state a chunk of 64
    tokens (the product and the power, 2), the powers themselves (the exponent g n log2 e with three
    roundings, while the power is above 2^-126: 3 x 126 ln 2 = 262), the sum over heads, and 32 for
    scales and joins."""
    return (dim + 64 + 2 * (tokens // 64 + 1) + 262 + group + 32) * 2.0 ** -24


def bounds(q, k, v, log_decay, scale, half_step, state=None, lengths=None, do=None, d_final=None, operands=None):
    """Element-wise error bounds of (o, states), or with ``do`` of (dq, dk, dv, dstate). Every result
    is a sum of products; with 16-bit operands (half_step 2^-8) the terms inside a chunk may carry the rounding
    of a score, those through the state that of the state's copy: ``operands`` bounds it, relative to the
    term (None: two roundings of 8 bits). The result is rounded once. States leave as sums of unrounded terms."""
    a = lambda x: None if x is None else np.abs(np.asarray(x, np.float64))  # noqa: E731
    T, D = q.shape[1], max(q.shape[3], v.shape[3])
    c32 = sums32(T, D, q.shape[2] // k.shape[2])
    if operands is None:
        operands = 2.02 * half_step
    rounded = c32 + (operands if half_step > 2.0 ** -24 else 0.0)
    tiny = 1e-37
    if do is None:
        o, S = forward(q, k, v, log_decay, scale, state, lengths)
        oa, Sa = forward(a(q), a(k), a(v), log_decay, abs(scale), a(state), lengths)
        return rounded * oa + 1.01 * half_step * np.abs(o) + tiny, c32 * Sa + tiny
    got = backward(do, q, k, v, log_decay, scale, state, lengths, d_final)
    top = backward(a(do), a(q), a(k), a(v), log_decay, abs(scale), a(state), lengths, a(d_final))
    return tuple(rounded * t + 1.01 * half_step * np.abs(r) + tiny for t, r in zip(top[:3], got[:3])) + (c32 * top[3] + tiny,)


def step(q, k, v, log_decay, scale, state):
    """(o, new states) of one token: q batch x heads x dim."""
    o, S = forward(q[:, None], k[:, None], v[:, None], log_decay, scale, state)
    return o[:, 0], S
