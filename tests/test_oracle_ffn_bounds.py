"""The error bounds of the feed-forward oracle: wide enough for the formulas evaluated in fp32,
too narrow for a wrong slope of a gate far outside the curved range."""

import numpy as np
import pytest

from oracle import ffn as of

ACTS = ["silu", "gelu_tanh"]


def fp32_forms(g, act):
    """(act(g), act'(g)) in fp32 steps: exponentials of a scaled argument, one reciprocal."""
    f = np.float32
    g = g.astype(f)
    log2e, one = f(1.4426950408889634), f(1.0)
    with np.errstate(over="ignore"):
        if act == "silu":
            s = one / (one + np.exp2(-g * log2e))
            return g * s, s * (one + g * (one - s))
        c, b = f(0.7978845608028654), f(0.044715)
        g2 = np.minimum(g * g, f(1e30))
        v = c * (g + b * g * g2)
        th = one - f(2.0) / (np.exp2(f(2.0) * log2e * v) + one)
        return f(0.5) * g * (one + th), f(0.5) * (one + th) + f(0.5) * g * (one - th * th) * c * (one + f(3.0) * b * g2)


@pytest.mark.parametrize("act", ACTS)
def test_fp32_activations_are_inside(act):
    g = np.concatenate([np.linspace(-40, 40, 400001), np.linspace(-3000, 3000, 60001)]).astype(np.float32)
    a, s = fp32_forms(g, act)
    want_a, want_s = of.activation(g.astype(np.float64), act)
    err_a, err_s = of.activation_errors(g.astype(np.float64), np.zeros(g.shape), act)
    assert np.all(np.abs(a - want_a) <= err_a) and np.all(np.abs(s - want_s) <= err_s)


@pytest.mark.parametrize("act", ACTS)
def test_wrong_slopes_of_far_gates_are_outside(act, monkeypatch):
    """Gates of some hundreds: a slope of 0.7 for 1, or of 0.3 for 0, leaves the bounds of dx and g_gate."""
    rng = np.random.default_rng(2)
    T, D, F = 20, 64, 64
    x, wg, wu, wd, dy = (s * rng.standard_normal(n) for n, s in (((T, D), 300.0), ((F, D), 0.25), ((F, D), 0.125),
                                                                ((D, F), 0.125), ((T, D), 0.5)))
    ops = (x, wg, wu, wd)
    want = of.backward(dy, *ops, act)
    bound = of.bounds(*ops, act, 2.0 ** -24, dy)
    true = of.activation

    def wrong(g, act):
        a, s = true(g, act)
        far = np.abs(g) > 100.0
        return a, np.where(far & (s > 0.5), 0.7, np.where(far, 0.3, s))
    monkeypatch.setattr(of, "activation", wrong)
    got = of.backward(dy, *ops, act)
    for k, name in ((0, "dx"), (1, "g_gate")):
        assert np.mean(np.abs(got[k] - want[k]) > bound[k]) > 0.9, name
    for k in (2, 3):        # du and h do not use the slope
        assert np.all(np.abs(got[k] - want[k]) <= bound[k])
