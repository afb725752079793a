"""Pins of the float64 oracles of a layer's operators (oracle/mixer.py, experts.py, dropout.py)."""

import numpy as np
import pytest

from oracle import dropout as od
from oracle import experts as oe
from oracle import mixer as om


def draw(seed, B, T, H, kv, D, E):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    return n((B, T, H, D)), n((B, T, kv, D)), n((B, T, kv, E)), n((B, T, H, E)), -np.geomspace(1.0, 0.01, H), n((B, H, D, E)), n((B, H, D, E))


def test_attention_is_its_double_sum():
    """o_i = scale (sum_{j <= i} e^{g (i - j)} (q_i . k_j) v_j + e^{g (i + 1)} q_i S_0) written out."""
    q, k, v, _, g, s, _ = draw(0, 2, 9, 4, 2, 3, 5)
    o, last = om.forward(q, k, v, g, 0.7, s)
    for b in range(2):
        for h in range(4):
            for i in range(9):
                want = np.exp(g[h] * (i + 1)) * q[b, i, h] @ s[b, h]
                for j in range(i + 1):
                    want = want + np.exp(g[h] * (i - j)) * (q[b, i, h] @ k[b, j, h // 2]) * v[b, j, h // 2]
                assert np.allclose(o[b, i, h], 0.7 * want, rtol=1e-12, atol=1e-12)
            want = np.exp(9 * g[h]) * s[b, h] + sum(np.exp(g[h] * (8 - j)) * np.outer(k[b, j, h // 2], v[b, j, h // 2]) for j in range(9))
            assert np.allclose(last[b, h], want, rtol=1e-12, atol=1e-12)


def test_attention_without_decay_counts():
    """Ones everywhere, no decay: o_i = scale dim (i + 1)."""
    one = np.ones((1, 6, 1, 4))
    o, last = om.forward(one, one, one, [0.0], 0.5)
    assert np.array_equal(o[0, :, 0], np.repeat(2.0 * np.arange(1, 7)[:, None], 4, 1)) and np.all(last == 6.0)
    o, _ = om.forward(one, one, one, [-np.inf], 0.5)       # and with nothing kept: the token alone
    assert np.all(o == 2.0)


@pytest.mark.parametrize("lengths", [None, [5, 0]])
def test_attention_gradients_are_differences(lengths):
    q, k, v, do, g, s, df = draw(1, 2, 7, 4, 2, 3, 2)
    value = lambda *a: sum(float((x * y).sum()) for x, y in zip(om.forward(*a[:3], g, 0.7, a[3], lengths), (do, df)))  # noqa: E731
    # an output behind a sequence is zero whatever comes
    grads = om.backward(do, q, k, v, g, 0.7, s, lengths, df)
    ops, rng = [q, k, v, s], np.random.default_rng(2)
    for i in range(4):
        move = rng.standard_normal(ops[i].shape)
        up, down = list(ops), list(ops)
        up[i], down[i] = ops[i] + move, ops[i] - move
        # linear in each operand alone: the difference is exact
        assert np.isclose((value(*up) - value(*down)) / 2, float((grads[i] * move).sum()), rtol=1e-10, atol=1e-10)


def test_attention_bounds_hold_for_rounded_operands():
    """A bound covers the rounding of what it names: scores rounded to 8 bits, result rounded."""
    q, k, v, _, g, _, _ = draw(3, 1, 40, 2, 2, 8, 8)
    r = lambda x: np.round(x / 2.0 ** (np.floor(np.log2(np.abs(x) + 1e-300)) - 7)) * 2.0 ** (np.floor(np.log2(np.abs(x) + 1e-300)) - 7)  # noqa: E731
    want, _ = om.forward(q, k, v, g, 1.0)
    i = np.arange(40)
    p = np.where(i[:, None] >= i[None, :], np.exp(g[:, None, None] * np.maximum(i[:, None] - i[None, :], 0)), 0.0)
    scores = np.einsum("ihd,jhd->hij", q[0], k[0]) * p
    got = np.einsum("hij,jhe->ihe", r(scores), v[0])
    limit, _ = om.bounds(q, k, v, g, 1.0, 2.0 ** -8)
    assert np.all(np.abs(r(got) - want[0]) <= limit[0])


def test_plan_and_rows_by_hand():
    ids = np.array([[2, 0], [-1, 2], [0, 5]])
    order, slots, offsets = oe.plan(ids, 4)
    assert order.tolist() == [1, 4, 0, 3, -1, -1] and slots.tolist() == [[2, 0], [-1, 3], [1, -1]] and offsets.tolist() == [0, 2, 2, 4, 4]
    x = np.array([[1.0], [2.0], [3.0]])
    xs = oe.dispatch(x, order, 2)
    assert xs[:, 0].tolist() == [1.0, 3.0, 1.0, 2.0, 0.0, 0.0]
    w = np.array([[10.0, 100.0], [7.0, 0.5], [1.0, 9.0]])
    y, _ = oe.combine(xs, w, slots)
    assert y[:, 0].tolist() == [110.0, 1.0, 3.0]
    # its gradients by differences: bilinear in rows and weights
    rng = np.random.default_rng(0)
    ys, dy = rng.standard_normal((6, 3)), rng.standard_normal((3, 3))
    dys, dw, _ = oe.combine_backward(dy, ys, w, slots)
    value = lambda a, b: float((oe.combine(a, b, slots)[0] * dy).sum())  # noqa: E731
    m, n = rng.standard_normal(ys.shape), rng.standard_normal(w.shape)
    assert np.isclose((value(ys + m, w) - value(ys - m, w)) / 2, (dys * m).sum())
    assert np.isclose((value(ys, w + n) - value(ys, w - n)) / 2, (dw * n).sum())


def test_philox_known_answers():
    """The known answers that its authors publish beside the generator: zeros, ones, digits of pi."""
    hexes = lambda s: [int(x, 16) for x in s.split()]  # noqa: E731
    for counter, key, want in [("0 0 0 0", "0 0", "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
                               ("ffffffff ffffffff ffffffff ffffffff", "ffffffff ffffffff", "408f276d 41c83b0e a20bc7c6 6d5451fd"),
                               ("243f6a88 85a308d3 13198a2e 03707344", "a4093822 299f31d0", "d16cfe09 94fdcceb 5001e420 24126ea1")]:
        assert od.philox(hexes(counter), hexes(key)) == hexes(want)


def test_dropout_keeps_its_share():
    x = np.ones(80000)
    for p in (0.1, 0.5):
        y = od.dropout(x, p, 1, 2)
        c = od.threshold(p)
        keep = 1 - c / 65536
        assert set(np.unique(y)) == {0.0, 65536.0 / (65536 - c)}
        assert abs((y != 0).mean() - keep) <= 6 * np.sqrt(keep * (1 - keep) / x.size)
    a, b = od.dropout(x, 0.5, 1, 2) != 0, od.dropout(x, 0.5, 1, 3) != 0
    assert abs((a == b).mean() - 0.5) <= 6 * 0.5 / np.sqrt(x.size)   # another offset, another mask
    assert od.threshold(0.0) == 0 and od.threshold(1.0) == 65536 and np.all(od.dropout(x, 1.0, 1, 2) == 0)
