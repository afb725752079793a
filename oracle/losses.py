"""Losses over vocabulary logits in NumPy float64, with their gradients, from the formulas:

    z = logits / tau, q = softmax(z), lse = log sum exp z
    policy:  lp = z_t - lse, rho = exp(lp - old),
             l = -min(rho A, clip(rho, 1 - cl, 1 + ch) A) + beta (exp(ref - lp) - (ref - lp) - 1)
    distill: p_j = exp(t_j / tau - L), l = sum_j p_j (log p_j - (z_{i_j} - lse))

Rows of weight 0 (or without a target) take no part. Each function also returns how far an
fp32 evaluation whose gradient is rounded to a storage type may be off, element by element.
"""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def _softmax(z):
    with np.errstate(invalid="ignore", over="ignore"):
        m = z.max()
        e = np.exp(z - m)
        s = e.sum()
        return m, e / s, np.log(s)


def _normaliser_error(z, q, m, lse, lse_given):
    """Errors of the normaliser: of lse as one float; of log q_v by what the normaliser
    contributes; relative, of each q_v. The fp32 difference z - m, its product with the scale
    (itself rounded) and the exponential's argument each carry 2^-24 of |z - m|; the
    exponential and the sums (at most V / 256 terms in a chain, and the joins) a few 2^-24
    more; neither |z| nor |lse| enters. lse_given: lse is read as one float, whose own
    rounding, and that of its product with the temperature, counts in every difference z - lse."""
    with np.errstate(invalid="ignore"):
        far = np.where(q > 0, np.abs(z - m), 0.0)
        off = np.where(q > 0, np.abs(z - lse), 0.0)
    s_err = U * (4.0 * float((q * far).sum()) + z.size / 256 + 60.0)
    lse_err = s_err + U * (4.0 * abs(lse) + 4.0 * abs(m))
    if lse_given:
        one = lse_err + 3.0 * U * abs(lse)
        return lse_err, one, one + U * (5.0 * off + 8.0)
    return lse_err, s_err, s_err + U * (4.0 * far + 8.0)


def policy(logits, targets, old, adv, ref=None, weights=None, grad_rows=None, *, clip_low, clip_high, kl_coef,
           temperature, half_step, lse_given=False):
    """Dict of loss, logp, lse, grad and err_loss, err_logp, err_lse, err_grad."""
    n, V = logits.shape
    out = {k: np.zeros(n) for k in ("loss", "logp", "lse", "err_loss", "err_logp", "err_lse")}
    out["grad"], out["err_grad"] = np.zeros((n, V)), np.zeros((n, V))
    for r in range(n):
        w = 1.0 if weights is None else float(weights[r])
        t = int(targets[r])
        if w == 0.0 or not 0 <= t < V:
            continue
        up = 1.0 if grad_rows is None else float(grad_rows[r])
        z = np.asarray(logits[r], np.float64) / temperature
        m, q, logs = _softmax(z)
        lse = m + logs
        e_lse, e_norm, e_q = _normaliser_error(z, q, m, lse, lse_given)
        lp = (z[t] - m) - logs   # not z_t - lse: m may be the type's lowest value
        # (z_t - m) c: five roundings of |z_t - m|; log2 s (at most |lp|) two, the difference and
        # its product with ln 2 three of |lp|
        e_lp = e_norm + U * (6.0 * abs(z[t] - m) + 6.0 * abs(lp))
        A, d_old = float(adv[r]), lp - float(old[r])
        rho = np.exp(d_old)
        cut = min(max(rho, 1.0 - clip_low), 1.0 + clip_high)
        kept = rho * A <= cut * A
        l = -(rho if kept else cut) * A
        slope = -rho * A if kept else 0.0
        e_rho = rho * (e_lp + U * (4.0 * abs(d_old) + 4.0))
        e_l = abs(A) * e_rho + 4.0 * U * abs(l)
        e_slope = (abs(A) * e_rho + 4.0 * U * abs(slope)) if kept else 0.0
        if kl_coef:
            d = float(ref[r]) - lp
            em1 = np.expm1(d)
            l += kl_coef * (em1 - d)
            slope += -kl_coef * em1
            e_em1 = np.exp(d) * (e_lp + U * (4.0 * abs(d) + 8.0)) + 4.0 * U * abs(em1)
            e_l += kl_coef * (e_em1 + e_lp + 4.0 * U * (abs(em1) + abs(d))) + 2.0 * U * abs(l)
            e_slope += kl_coef * e_em1 + 2.0 * U * abs(slope)
        scale = w * up / temperature
        hot = np.zeros(V)
        hot[t] = 1.0
        g = scale * slope * (hot - q)
        out["loss"][r], out["logp"][r], out["lse"][r], out["grad"][r] = w * l, lp, lse, g
        out["err_loss"][r] = abs(w) * e_l + 2.0 * U * abs(w * l)
        out["err_logp"][r], out["err_lse"][r] = e_lp, e_lse
        out["err_grad"][r] = (abs(scale) * (e_slope * np.abs(hot - q) + abs(slope) * (q * e_q + 4.0 * U * (hot + q)))
                              + half_step * np.abs(g) + 1e-38)
    return out


def distill(logits, top, ids, top_lse=None, weights=None, grad_rows=None, *, temperature, half_step, lse_given=False):
    """Dict of loss, lse, grad and err_loss, err_lse, err_grad."""
    n, V = logits.shape
    out = {k: np.zeros(n) for k in ("loss", "lse", "err_loss", "err_lse")}
    out["grad"], out["err_grad"] = np.zeros((n, V)), np.zeros((n, V))
    for r in range(n):
        w = 1.0 if weights is None else float(weights[r])
        if w == 0.0:
            continue
        up = 1.0 if grad_rows is None else float(grad_rows[r])
        z = np.asarray(logits[r], np.float64) / temperature
        m, q, logs = _softmax(z)
        lse = m + logs
        e_lse, e_norm, e_q = _normaliser_error(z, q, m, lse, lse_given)
        there = (ids[r] >= 0) & (ids[r] < V) & (top[r] > -np.inf)
        at = ids[r][there].astype(int)
        t = np.asarray(top[r], np.float64)[there] / temperature
        l = mass = e_l = e_mass = 0.0
        pv, e_pv = np.zeros(V), np.zeros(V)
        if t.size:
            norm = t.max() + np.log(np.exp(t - t.max()).sum()) if top_lse is None else float(top_lse[r])
            lp = t - norm
            p = np.exp(lp)
            # the arguments' roundings, the normaliser's (over the kept entries) and the exponential's
            e_lp = U * (6.0 * np.abs(t - t.max()) + 6.0 * np.abs(lp) + 8.0 * np.abs(t).max() + 8.0 * abs(norm)
                        + t.size / 64 + 60.0)
            e_p = p * (e_lp + 4.0 * U)
            lq = (z[at] - m) - logs
            e_lq = e_norm + U * (6.0 * np.abs(z[at] - m) + 6.0 * np.abs(lq))
            terms = p * (lp - lq)
            l, mass = terms.sum(), p.sum()
            e_l = (e_p * np.abs(lp - lq) + p * (e_lp + e_lq) + 8.0 * U * p * (np.abs(lp) + np.abs(lq))).sum()
            e_l += (t.size / 64 + 20) * U * np.abs(terms).sum()
            e_mass = e_p.sum() + (t.size / 64 + 20) * U * mass
            np.add.at(pv, at, p)
            np.add.at(e_pv, at, e_p + p * t.size * U)
        scale = w * up / temperature
        g = scale * (mass * q - pv)
        out["loss"][r], out["lse"][r], out["grad"][r] = w * l, lse, g
        out["err_loss"][r] = abs(w) * e_l + 4.0 * U * abs(w * l)
        out["err_lse"][r] = e_lse
        out["err_grad"][r] = (abs(scale) * (q * e_mass + mass * q * (e_q + 6.0 * U) + e_pv + 4.0 * U * pv)
                              + half_step * np.abs(g) + 1e-38)
    return out
