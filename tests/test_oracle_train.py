"""Pins of the feed-forward and loss oracles: gradients against central differences, an
independent float64 implementation (torch on the CPU), and closed forms."""

import numpy as np
import pytest
import torch

from oracle import ffn as of
from oracle import losses as ol


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_ffn_gradients_match_differences(act):
    rng = np.random.default_rng(3)
    T, D, F = 4, 5, 7
    ops = [rng.standard_normal(s) for s in ((T, D), (F, D), (F, D), (D, F))]
    dy = rng.standard_normal((T, D))
    grads = of.backward(dy, *ops, act)
    step = 1e-5   # error of a central difference: step^2 / 6 f''' + 1e-16 / step, well under 1e-7
    for k, g in enumerate(grads):
        for at in [(0, 0), (1, 2), (g.shape[0] - 1, g.shape[1] - 1)]:
            up = [o.copy() for o in ops]
            down = [o.copy() for o in ops]
            up[k][at] += step
            down[k][at] -= step
            diff = ((of.forward(*up, act) - of.forward(*down, act)) * dy).sum() / (2 * step)
            assert abs(diff - g[at]) <= 1e-7 * max(1.0, abs(g[at])), (k, at)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_ffn_matches_torch_float64(act):
    rng = np.random.default_rng(4)
    x, wg, wu, wd = (torch.from_numpy(rng.standard_normal(s)) for s in ((6, 8), (10, 8), (10, 8), (8, 10)))
    f = torch.nn.functional
    gate = x @ wg.T
    gate = f.silu(gate) if act == "silu" else f.gelu(gate, approximate="tanh")
    y = (gate * (x @ wu.T)) @ wd.T
    assert np.allclose(of.forward(x, wg, wu, wd, act), y.numpy(), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_activation_slope_bounds(act):
    """The slopes of act and act' used by the error bounds."""
    g = np.linspace(-30, 30, 200001)
    a, s = of.activation(g, act)
    assert np.abs(np.diff(a) / np.diff(g)).max() <= 1.13
    assert np.abs(np.diff(s) / np.diff(g)).max() <= 1.13


def policy_inputs(rng, n, V):
    z = 2.0 * rng.standard_normal((n, V))
    t = rng.integers(0, V, n)
    lp = np.array([z[r, t[r]] - np.log(np.exp(z[r]).sum()) for r in range(n)])
    return z, t, lp - rng.uniform(-0.6, 0.6, n), rng.standard_normal(n), lp + 0.3 * rng.standard_normal(n)


def test_policy_gradient_matches_differences():
    rng = np.random.default_rng(5)
    n, V = 6, 11
    z, t, old, adv, ref = policy_inputs(rng, n, V)
    w, up = rng.uniform(0.5, 2, n), rng.standard_normal(n)
    kw = dict(clip_low=0.2, clip_high=0.3, kl_coef=0.1, temperature=1.3, half_step=0.0)
    run = lambda a: ol.policy(a, t, old, adv, ref, w, up, **kw)  # noqa: E731
    got = run(z)
    step = 1e-5
    for r in range(n):
        for v in range(V):
            hi, lo = z.copy(), z.copy()
            hi[r, v] += step
            lo[r, v] -= step
            diff = up[r] * (run(hi)["loss"][r] - run(lo)["loss"][r]) / (2 * step)
            assert abs(diff - got["grad"][r, v]) <= 1e-7, (r, v)


@pytest.mark.parametrize("given", [False, True])
def test_distill_gradient_matches_differences(given):
    rng = np.random.default_rng(6)
    n, V, K = 5, 13, 4
    z, top = 2.0 * rng.standard_normal((n, V)), 3.0 * rng.standard_normal((n, K))
    ids = np.stack([rng.permutation(V)[:K] for _ in range(n)])
    ids[1, 2] = -1          # absent
    ids[2, 1] = ids[2, 0]   # the same column twice
    tau = 1.7
    lse = np.log(np.exp(top / tau).sum(1)) + 0.3 if given else None
    run = lambda a: ol.distill(a, top, ids, lse, temperature=tau, half_step=0.0)  # noqa: E731
    got = run(z)
    step = 1e-5
    for r in range(n):
        for v in range(V):
            hi, lo = z.copy(), z.copy()
            hi[r, v] += step
            lo[r, v] -= step
            diff = (run(hi)["loss"][r] - run(lo)["loss"][r]) / (2 * step)
            assert abs(diff - got["grad"][r, v]) <= 1e-7, (r, v)


def test_policy_closed_forms():
    rng = np.random.default_rng(7)
    z, t, _, adv, _ = policy_inputs(rng, 4, 9)
    kw = dict(clip_low=0.2, clip_high=0.2, kl_coef=0.5, temperature=1.0, half_step=0.0)
    lp = ol.policy(z, t, np.zeros(4), adv, np.zeros(4), **kw)["logp"]
    # the old, the reference and the new policy agree: loss -A, gradient A (q - onehot)
    got = ol.policy(z, t, lp, adv, lp, **kw)
    assert np.allclose(got["loss"], -adv)
    q = np.exp(z - np.log(np.exp(z).sum(1))[:, None])
    hot = np.eye(9)[t]
    assert np.allclose(got["grad"], adv[:, None] * (q - hot))
    # without a target a row takes no part
    assert not ol.policy(z, np.full(4, -100), lp, adv, lp, **kw)["grad"].any()


def test_distill_of_the_teacher_itself_is_zero():
    """All entries kept and equal to the student's logits: loss 0, gradient 0."""
    rng = np.random.default_rng(8)
    z = rng.standard_normal((3, 10))
    ids = np.tile(np.arange(10), (3, 1))
    got = ol.distill(z, z, ids, temperature=2.0, half_step=0.0)
    assert np.abs(got["loss"]).max() < 1e-14 and np.abs(got["grad"]).max() < 1e-15
