"""How exact linear attention with decay is: the error of bf16 results against float64, as a multiple of the
error that rounding the float64 results once to bf16 makes."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import mixer as om  # noqa: E402
from tests.gpu_util import TORCH_DT, rel, to_np  # noqa: E402


@pytest.fixture(scope="module")
def X():
    from matrix_orthogonalising_optimizer_muon_amd import mixers
    return mixers


def inputs(B, T, H, kv, D, E, dtype):
    """Random operands and states, decays slow enough that what is carried over chunks counts."""
    rng = np.random.default_rng([7, B, T, H, D, E])
    new = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).cuda()  # noqa: E731
    q, k, v, do = (new(B, T, h, d).to(TORCH_DT[dtype]) for h, d in ((H, D), (kv, D), (kv, E), (H, E)))
    g = torch.from_numpy(-np.geomspace(0.03, 2e-4, H).astype(np.float32)).cuda()
    return q, k, v, do, g, new(B, H, D, E) * 8.0, new(B, H, D, E) * 8.0


def group_of(ins, b, j):
    """Sequence b and the query heads of k, v head j alone, as float64 arrays, and their slices of results."""
    q, k, v, do, g, s, df = ins
    n = q.shape[2] // k.shape[2]
    heads, one, at = slice(j * n, (j + 1) * n), slice(j, j + 1), slice(b, b + 1)
    a = [to_np(t) for t in (q[at, :, heads], k[at, :, one], v[at, :, one], g[heads])]
    per_token = {"o": heads, "dq": heads, "dk": one, "dv": one}
    pick = lambda t, name: to_np(t[at, heads] if name in ("states", "dstate") else t[at, :, per_token[name]])  # noqa: E731
    return a, to_np(do[at, :, heads]), to_np(s[at, heads]), to_np(df[at, heads]), pick


def results(X, ins, with_states):
    q, k, v, do, g, s, df = ins
    if not with_states:
        o, _ = X.linear_attention_forward(q, k, v, g)
        return dict(zip(("o", "dq", "dk", "dv"), (o, *X.linear_attention_backward(do, q, k, v, g)[:3])))
    o, last = X.linear_attention_forward(q, k, v, g, state=s, final=True)
    grads = X.linear_attention_backward(do, q, k, v, g, state=s, d_final=df, need_dstate=True)
    return dict(zip(("o", "states", "dq", "dk", "dv", "dstate"), (o, last, *grads)))


def exact(a, do, s, df, with_states):
    f = float(np.float32(1.0 / np.sqrt(a[0].shape[3])))
    s, df = (s, df) if with_states else (None, None)
    o, last = om.forward(*a, f, s)
    return dict(zip(("o", "states", "dq", "dk", "dv", "dstate"), (o, last, *om.backward(do, *a, f, s, None, df))))


# slices of 32, 64 and 128 columns, heads up to 256; rows of whole 16 bytes and others; one walk and segments
SIZES = [(64, 330, 4, 2, 128, 128), (64, 330, 4, 4, 126, 127), (32, 260, 4, 2, 256, 256), (32, 260, 2, 1, 250, 255),
         (1, 4100, 16, 8, 128, 128), (1, 4100, 16, 8, 127, 126), (1, 3000, 8, 4, 256, 256), (1, 3001, 8, 8, 249, 251),
         (64, 330, 4, 2, 64, 64), (1, 1500, 2, 1, 126, 127), (1, 1500, 2, 2, 33, 65), (1, 1500, 2, 2, 256, 256)]


@pytest.mark.parametrize("with_states", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_bf16_results_are_as_exact_as_one_rounding(X, size, with_states):
    """Operands that are rounded on the way have two parts of 8 bits, each wrong by at most 2^-17 of itself: a score, a weighted
    row, the state's copy. Random terms add up in quadrature, as the result does, so all of them make at most 3 x 2^-17 of its
    norm, where its own rounding makes about 0.42 x 2^-8 (uniform over the step, averaged over a binade): together
    sqrt(1 + (3 x 2^-9 / 0.42)^2) = 1.0001 times that. One of the three with one part: up to sqrt(1 + 1) times."""
    ins = inputs(*size, "bf16")
    got = results(X, ins, with_states)
    B, kv = size[0], size[3]
    ratios = {}
    for b, j in {(0, 0), (B - 1, kv - 1)}:
        a, do, s, df, pick = group_of(ins, b, j)
        for name, want in exact(a, do, s, df, with_states).items():
            if name in got and name not in ("states", "dstate"):
                once = torch.from_numpy(want).bfloat16().double().numpy()
                ratios[name, b, j] = rel(pick(got[name], name), want) / rel(once, want)
    print(size, with_states, {k: round(v, 4) for k, v in ratios.items()})
    assert max(ratios.values()) <= 1.01, ratios


def steps32(size, name):
    """A bound of the fp32 error's norm, relative to the result's, in steps of 2^-24: a sum of n random terms whose running
    sum is rounded after each has sqrt(n / 2) roundings' worth, each 0.42 of a half step (uniform over the step, averaged over a
    binade). How often a matrix instruction rounds is not documented; after each of its products at most: dim for a score
    and for a row through the state, 64 for a chunk's tokens in a score row's sum, 64 in the state's. The state
    takes one rounding for each chunk before it; eight more for powers, scales and joins. With products summed onto the state
    itself, each of its chunks' roundings would be of its size (and a power in one fp32 number would be wrong by up to a step,
    chunk after chunk the same way)."""
    B, T, H, kv, D, E = size
    dim = {"o": D, "dq": E, "dk": E, "dv": D}.get(name, 0)
    chunks, sums = -(-T // 64), 2 if dim else 1
    return 0.42 * np.sqrt(2 * dim / 2 + sums * 64 / 2 + chunks / 2 + (H // kv) / 2 + 8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES + [(8, 1540, 16, 8, 128, 128), (8, 1541, 16, 16, 63, 62), (4, 1100, 16, 8, 256, 256)])
def test_fp32_results_are_as_exact_as_sums_by_chunks(X, size, dtype):
    """fp32 results, and the states of bf16 operands, within the bound."""
    ins = inputs(*size, dtype)
    got = results(X, ins, True)
    B, kv = size[0], size[3]
    ratios = {}
    for b, j in {(0, 0), (B - 1, kv - 1)}:
        a, do, s, df, pick = group_of(ins, b, j)
        for name, want in exact(a, do, s, df, True).items():
            if dtype == "f32" or name in ("states", "dstate"):
                ratios[name, b, j] = rel(pick(got[name], name), want) / (steps32(size, name) * 2.0 ** -24)
    print(size, dtype, {k: round(float(v), 2) for k, v in ratios.items()})
    assert max(ratios.values()) <= 1.0, ratios


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(2, 330, 4, 2, 128, 128), (1, 1500, 2, 1, 126, 127), (1, 700, 2, 2, 64, 40), (8, 330, 8, 8, 200, 256)])
def test_a_state_that_leaves_changes_no_other_result(X, size, dtype):
    q, k, v, do, g, s, df = inputs(*size, dtype)
    for kw in ({}, dict(state=s)):
        assert torch.equal(X.linear_attention_forward(q, k, v, g, **kw)[0], X.linear_attention_forward(q, k, v, g, **kw, final=True)[0])
        a = X.linear_attention_backward(do, q, k, v, g, **kw, d_final=df)
        b = X.linear_attention_backward(do, q, k, v, g, **kw, d_final=df, need_dstate=True)
        assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))


def test_decay_does_not_drift_over_many_steps(X):
    """2048 tokens of zeros leave e^{2048 g} of a state. A rounding a step, as likely up as down: 0.42 sqrt(2048) = 19 steps of
    2^-24 in the norm, and 1.5 times that for the powers' rests; a decay of one fp32 number is wrong by up to a
    half step the same way every time, 1024 steps in the end."""
    n = 2048
    g = torch.tensor([-1e-4, -3e-4, -7e-4, -1.1e-3], device="cuda")
    q, k, v = torch.zeros(1, 4, 32, device="cuda"), torch.zeros(1, 4, 32, device="cuda"), torch.zeros(1, 4, 64, device="cuda")
    s0 = torch.randn(1, 4, 32, 64, device="cuda")
    s = s0.clone()
    for _ in range(n):
        X.linear_attention_step(q, k, v, g, s)
    for h in range(4):
        want = to_np(s0[0, h]) * np.exp(float(g[h]) * n)
        assert rel(to_np(s[0, h]), want) <= 1.5 * 0.42 * np.sqrt(n) * 2.0 ** -24, h
