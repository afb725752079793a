"""What the losses' threads hold of a row: one normaliser, to the last bit."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from matrix_orthogonalising_optimizer_muon_amd import losses
    return losses


def cuda(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)


@pytest.mark.parametrize("temperature", [1.0, 0.7])
@pytest.mark.parametrize("half", [350, 20000, 76032, 131073])
def test_equal_logits_have_equal_gradients(S, half, temperature):
    """A row of two equal halves: its columns are dealt with by different threads, which have to
    hold the same normaliser to the last bit."""
    rng = np.random.default_rng([7, half])
    z = cuda(np.tile(2.5 * rng.standard_normal((6, half)), (1, 2)).astype(np.float32))
    t = cuda(rng.integers(0, half, 6), torch.int64)
    lp = torch.log_softmax(z.double() / temperature, 1).gather(1, t[:, None])[:, 0]
    _, _, grad = S.policy_loss(z, t, (lp - 0.05).float(), cuda(rng.standard_normal(6)), temperature=temperature)
    a, b = grad[:, :half].clone(), grad[:, half:].clone()
    at = torch.arange(6, device="cuda")
    a[at, t], b[at, t] = 0.0, 0.0
    assert torch.equal(a, b)
    _, grad = S.distill_loss(z, cuda(rng.standard_normal((6, 3))), t[:, None].repeat(1, 3), temperature=temperature)
    a, b = grad[:, :half].clone(), grad[:, half:].clone()
    a[at, t], b[at, t] = 0.0, 0.0
    assert torch.equal(a, b)
