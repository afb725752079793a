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
