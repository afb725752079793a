"""Tokens sorted by expert and back, in float64 and plain loops (the formulas of ``muon_experts`` in
``include/muon.h``), and error bounds of the sums."""

from __future__ import annotations

import numpy as np


def plan(ids, experts):
    """(order, slots, offsets) of ids (tokens x top)."""
    flat = np.asarray(ids).reshape(-1)
    order, slots, offsets = np.full(flat.size, -1), np.full(flat.size, -1), [0]
    p = 0
    for e in range(experts):
        for f in np.flatnonzero(flat == e):
            order[p], slots[f] = f, p
            p += 1
        offsets.append(p)
    return order, slots.reshape(np.shape(ids)), np.array(offsets)


def dispatch(x, order, top):
    x = np.asarray(x, np.float64)
    out = np.zeros((order.size, x.shape[1]))
    for p, f in enumerate(order):
        if f >= 0:
            out[p] = x[f // top]
    return out


def combine(ys, weights, slots):
    """(y, sum of the absolute terms); weights None: 1."""
    ys = np.asarray(ys, np.float64)
    T, top = slots.shape
    y, size = np.zeros((T, ys.shape[1])), np.zeros((T, ys.shape[1]))
    for t in range(T):
        for j in range(top):
            if slots[t, j] >= 0:
                term = ys[slots[t, j]] * (1.0 if weights is None else float(weights[t, j]))
                y[t] += term
                size[t] += np.abs(term)
    return y, size


def combine_backward(dy, ys, weights, slots):
    """(dys, dweights, sum of the absolute terms of dweights)."""
    dy, ys = np.asarray(dy, np.float64), np.asarray(ys, np.float64)
    T, top = slots.shape
    dys, dw, size = np.zeros_like(ys), np.zeros((T, top)), np.zeros((T, top))
    for t in range(T):
        for j in range(top):
            s = slots[t, j]
            if s >= 0:
                dys[s] = dy[t] * (1.0 if weights is None else float(weights[t, j]))
                dw[t, j] = dy[t] @ ys[s]
                size[t, j] = np.abs(dy[t]) @ np.abs(ys[s])
    return dys, dw, size
