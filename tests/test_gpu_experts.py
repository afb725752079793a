"""Tokens sorted by expert and back (muon_expert_*) against the float64 oracle: the plan exactly,
rows exactly, sums within their derived errors."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import experts as oe  # noqa: E402
from tests.gpu_util import TORCH_DT, to_np  # noqa: E402

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def E():
    from matrix_orthogonalising_optimizer_muon_amd import experts
    return experts


def check_plan(E, ids, experts):
    plan = E.expert_plan(ids, experts)
    order, slots, offsets = oe.plan(ids.cpu().numpy(), experts)
    assert np.array_equal(plan.order.cpu().numpy(), order)
    assert np.array_equal(plan.slots.cpu().numpy(), slots)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    return plan, order, slots, offsets


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("size", [(1, 1, 1), (1, 8, 8), (3, 2, 5), (64, 1, 2), (65, 3, 7), (2048, 1, 64), (2049, 1, 64),
                                  (1000, 8, 64), (5000, 8, 256), (300000, 2, 1024), (40000, 7, 3), (1, 64, 1024)])
def test_plan(E, size, dtype):
    T, top, n = size
    rng = np.random.default_rng(list(size))
    ids = rng.integers(0, n, (T, top))
    check_plan(E, torch.from_numpy(ids).cuda().to(dtype), n)
    # choices that are dropped, experts that nobody chose, one expert for all
    ids[rng.random((T, top)) < 0.3] = rng.choice([-1, n, n + 7, -(1 << 31)])
    check_plan(E, torch.from_numpy(ids).cuda().to(dtype), n)
    check_plan(E, torch.full((T, top), n - 1, device="cuda", dtype=dtype), n)
    check_plan(E, torch.full((T, top), -1, device="cuda", dtype=dtype), n)
    check_plan(E, torch.from_numpy(np.sort(rng.integers(0, max(n // 2, 1), T * top)).reshape(T, top)).cuda().to(dtype), n)


def test_plan_of_nothing_and_of_any_shape(E):
    plan = E.expert_plan(torch.empty(0, 2, dtype=torch.int64, device="cuda"), 5)
    assert plan.offsets.tolist() == [0] * 6 and plan.order.numel() == 0
    x = torch.empty(0, 8, device="cuda")
    assert E.dispatch_forward(x, plan).shape == (0, 8) and E.combine_forward(x, None, plan).shape == (0, 8)
    ids = torch.randint(0, 9, (2, 3, 4), device="cuda")
    plan = E.expert_plan(ids, 9)
    assert plan.slots.shape == ids.shape and plan.tokens == 6
    x = torch.randn(2, 3, 5, device="cuda")
    xs = E.dispatch_forward(x, plan)
    assert E.combine_forward(xs, None, plan).shape == x.shape
    assert torch.equal(E.expert_plan(ids[..., 0].contiguous(), 9).slots, E.expert_plan(ids[..., 0].contiguous().int(), 9).slots)
    big = torch.tensor([[1 << 32, 3]], device="cuda")     # outside, though its low word is 0
    assert E.expert_plan(big, 4).slots.tolist() == [[-1, 0]]


def rounded(rng, *shape, dtype, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).cuda().to(TORCH_DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(1, 1, 1, 1), (5, 2, 3, 7), (33, 3, 8, 64), (70, 8, 16, 127), (20, 5, 40, 520), (9, 1, 4, 2051),
                                  (12, 64, 70, 16), (130, 2, 6, 4099)])
@pytest.mark.parametrize("dropped", [0.0, 0.4, 1.0])
def test_rows(E, size, dtype, dropped):
    T, top, n, D = size
    rng = np.random.default_rng([*size, int(10 * dropped)])
    ids = np.stack([rng.permutation(max(n, top))[:top] for _ in range(T)]) % n
    ids[rng.random(ids.shape) < dropped] = -1
    plan, order, slots, offsets = check_plan(E, torch.from_numpy(ids).cuda(), n)
    x, ys, dy = rounded(rng, T, D, dtype=dtype), rounded(rng, T * top, D, dtype=dtype), rounded(rng, T, D, dtype=dtype)
    w = torch.from_numpy(rng.standard_normal((T, top)).astype(np.float32)).cuda()
    # what has no row is not read
    ys[int(offsets[-1]):] = float("nan")
    w[plan.slots < 0] = float("nan")
    h = HALF_STEP[dtype]
    clean = np.nan_to_num(to_np(ys))
    wn = np.where(slots >= 0, np.nan_to_num(to_np(w)), 0)
    assert np.array_equal(to_np(E.dispatch_forward(x, plan)), oe.dispatch(to_np(x), order, top))
    for weights, wa in ((w, wn), (None, None)):
        y, size_y = oe.combine(clean, wa, slots)
        err = 1.01 * h * np.abs(y) + (top + 2) * 2.0 ** -24 * size_y
        assert np.all(np.abs(to_np(E.combine_forward(ys, weights, plan)) - y) <= err)
        dys, dw, size_w = oe.combine_backward(to_np(dy), clean, wa, slots)
        got = E.combine_backward(dy, ys, weights, plan)
        assert np.all(np.abs(to_np(got[0]) - dys) <= (1.01 * h + 2.0 ** -24) * np.abs(dys))
        assert np.all(np.abs(to_np(got[1]) - dw) <= (D + 2) * 2.0 ** -24 * size_w)
        assert E.combine_backward(dy, None, weights, plan, need=(True, False))[1] is None
        assert torch.equal(E.combine_backward(dy, ys, weights, plan, need=(False, True))[1], got[1])
        assert torch.equal(E.combine_backward(dy, None, weights, plan, need=(True, False))[0], got[0])
    # dispatch's gradient is the sum of the rows
    assert torch.equal(E.dispatch_backward(ys, plan), E.combine_forward(ys, None, plan))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off,extra", [(0, 1), (1, 0), (8, 24), (3, 5)])
def test_rows_inside_wider_arrays(E, dtype, off, extra):
    rng = np.random.default_rng(off)
    T, top, n, D = 40, 3, 5, 101
    ids = torch.from_numpy(rng.integers(-1, n, (T, top))).cuda()
    plan = E.expert_plan(ids, n)
    w = torch.randn(T, top, device="cuda")

    def wide(t):
        b = torch.full((t.shape[0] + 2, off + D + extra), float("nan"), dtype=t.dtype, device="cuda")
        b[1:-1, off:off + D] = t
        return b[1:-1, off:off + D]
    x, ys, dy = (rounded(rng, r, D, dtype=dtype) for r in (T, T * top, T))
    assert torch.equal(E.dispatch_forward(wide(x), plan), E.dispatch_forward(x, plan))
    assert torch.equal(E.combine_forward(wide(ys), w, plan), E.combine_forward(ys, w, plan))
    for a, b in zip(E.combine_backward(wide(dy), wide(ys), w, plan), E.combine_backward(dy, ys, w, plan)):
        assert torch.equal(a, b)


def test_an_expert_twice(E):
    """A token that names one expert twice has two rows there; both count."""
    ids = torch.tensor([[2, 2], [0, 2]], device="cuda")
    plan, *_ = check_plan(E, ids, 3)
    ys = torch.arange(8.0, device="cuda").view(4, 2)
    w = torch.tensor([[1.0, 10.0], [100.0, 1000.0]], device="cuda")
    # rows: (1, 0), (0, 0), (0, 1), (1, 1)
    assert E.combine_forward(ys, w, plan).tolist() == [[2.0 + 40.0, 3.0 + 50.0], [0.0 + 6000.0, 100.0 + 7000.0]]


def test_automatic_differentiation(E):
    rng = np.random.default_rng(1)
    T, top, n, D = 30, 3, 6, 20
    plan = E.expert_plan(torch.from_numpy(rng.integers(-1, n, (T, top))).cuda(), n)
    x = torch.randn(5, 6, D, device="cuda", requires_grad=True)
    w = torch.rand(T, top, device="cuda", requires_grad=True)
    xs = E.dispatch(x, plan)
    ys = torch.tanh(xs)
    y = E.combine(ys, w, plan)
    gx, gw = torch.autograd.grad(y.sum(), (x, w))
    # the same in torch's operations
    xr, wr = x.detach().double().requires_grad_(True), w.detach().double().requires_grad_(True)
    there = (plan.slots >= 0).double()
    t = torch.tanh(xr.view(T, D))
    want = (t * (wr * there).sum(1, keepdim=True))
    rx, rw = torch.autograd.grad(want.sum(), (xr, wr))
    # sums of 3 terms below 1 of weight, of tanh's derivative of an fp32 tanh: some steps of 2^-24 of 3; of 20 terms
    assert float((gx.double() - rx).abs().max()) <= 3 * 16 * 2.0 ** -24
    assert float((gw.double() - rw).abs().max()) <= 20 * 32 * 2.0 ** -24
    # one of the two, neither weights
    assert torch.equal(torch.autograd.grad(E.combine(ys.detach(), w, plan).sum(), w)[0], gw)
    leaf = ys.detach().requires_grad_(True)
    assert torch.equal(torch.autograd.grad(E.combine(leaf, None, plan).sum(), leaf)[0],
                       E.combine_backward(torch.ones(T, D, device="cuda"), None, None, plan, need=(True, False))[0])


def test_refusals(E):
    ids = torch.randint(0, 4, (6, 2), device="cuda")
    plan = E.expert_plan(ids, 4)
    x, ys, w = torch.randn(6, 8, device="cuda"), torch.randn(12, 8, device="cuda"), torch.rand(6, 2, device="cuda")
    for bad, kind in [(lambda: E.expert_plan(ids.float(), 4), TypeError), (lambda: E.expert_plan(ids.cpu(), 4), ValueError),
                      (lambda: E.expert_plan(ids, 0), ValueError), (lambda: E.expert_plan(ids, 1025), ValueError),
                      (lambda: E.expert_plan(ids.t(), 4), ValueError),
                      (lambda: E.expert_plan(torch.zeros(2, 65, dtype=torch.int64, device="cuda"), 4), ValueError),
                      (lambda: E.expert_plan(torch.zeros(2, 0, dtype=torch.int64, device="cuda"), 4), ValueError),
                      (lambda: E.dispatch_forward(x[:5], plan), ValueError), (lambda: E.dispatch_forward(x.half(), plan), TypeError),
                      (lambda: E.dispatch_forward(x, ids), TypeError), (lambda: E.dispatch_forward(x.cpu(), plan), ValueError),
                      (lambda: E.combine_forward(x, w, plan), ValueError), (lambda: E.combine_forward(ys, w[:5], plan), ValueError),
                      (lambda: E.combine_forward(ys, w.double(), plan), TypeError),
                      (lambda: E.combine_forward(ys, w.t(), plan), ValueError),
                      (lambda: E.combine_backward(x, ys[:, :4], w, plan), ValueError),
                      (lambda: E.combine_backward(x, ys.bfloat16(), w, plan), TypeError),
                      (lambda: E.combine_backward(x, None, w, plan), TypeError),
                      (lambda: E.RoutedFeedForward(8, 8, 4, 5, device="cuda"), ValueError)]:
        with pytest.raises(kind):
            bad()
