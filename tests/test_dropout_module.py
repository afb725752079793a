"""The Dropout module's numbers, on the CPU: the mask is the oracle's, in place of the kernel."""

import numpy as np
import pytest
import torch
from torch.utils.checkpoint import checkpoint

from oracle import dropout as od

R = pytest.importorskip("matrix_orthogonalising_optimizer_muon_amd.dropout")


@pytest.fixture(autouse=True)
def oracle_mask(monkeypatch):
    def call(x, p, seed, offset, residual, out):
        if isinstance(seed, torch.Tensor):
            seed, offset = (int(n) % (1 << 64) for n in seed)
        keep = od.numbers(x.numel(), seed, offset) >= od.threshold(p)
        y = x * torch.from_numpy(keep.reshape(x.shape).astype(np.float32)).to(x.dtype)
        return y if residual is None else y + residual
    monkeypatch.setattr(R, "_call", call)


def run(m, x, how, **kw):
    """The mask of an output and that of its gradient, the module's call being run again in the backward or not."""
    leaf = x.clone().requires_grad_(True)
    y = m(leaf) if how is None else checkpoint(m, leaf, use_reentrant=how, **kw)
    g, = torch.autograd.grad(y.sum(), leaf) if how is not True else [(y.sum().backward(), leaf.grad)[1]]
    return y.detach() != 0, g != 0


@pytest.mark.parametrize("reentrant", [False, True])
def test_counted_calls_are_not_run_again(reentrant):
    """A count of calls has gone on when a checkpointed forward runs again: another mask than the loss saw. Refused."""
    m, x = R.Dropout(0.5, seed=3), torch.ones(40, 10)
    a, b = run(m, x, None)
    assert torch.equal(a, b) and m.counter.tolist() == [3, 1]
    with pytest.raises(RuntimeError, match="counts its calls"):
        run(m, x, reentrant)
    assert m.counter.tolist() == [3, 2]
    # the call with numbers of its own runs again as it was
    a, b = run(lambda t: R.dropout(t, 0.5, 3, 7), x, reentrant)
    assert torch.equal(a, b)


def test_modules_draw_masks_of_their_own():
    """Built alike, copied, called again: another mask each, and the same ones after torch.manual_seed."""
    import copy
    x = torch.ones(50, 20)

    def masks():
        torch.manual_seed(5)
        first, second = R.Dropout(0.5), R.Dropout(0.5)
        return [m(x) != 0 for m in (first, second, copy.deepcopy(first), first)]
    one, two = masks(), masks()
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    for i in range(4):
        for j in range(i):
            # 1000 coins of 1/2: six deviations
            assert abs(float((one[i] == one[j]).float().mean()) - 0.5) <= 6 * 0.5 / np.sqrt(1000), (i, j)


@pytest.mark.parametrize("reentrant", [False, True])
def test_a_checkpointed_call_draws_its_mask_again(reentrant):
    m, x = R.Dropout(0.5), torch.ones(40, 10)
    torch.manual_seed(6)
    a, b = run(m, x, None)
    torch.manual_seed(6)
    c, d = run(m, x, reentrant)
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)


def test_seed_and_state():
    assert R.Dropout(0.1).counter is None and list(R.Dropout(0.1).state_dict()) == []
    m = R.Dropout(0.1, seed=-2)
    m(torch.ones(3))
    other = R.Dropout(0.1, seed=9)
    other.load_state_dict(m.state_dict())
    assert other.counter.tolist() == [-2, 1]
    assert torch.equal(R.Dropout(0.0)(x := torch.ones(3)), x) and torch.equal(R.Dropout(0.5).eval()(x, x), 2 * x)
