"""DecayAttention after a cast does what one built in that type does."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_cast_module_runs_as_one_built_in_bf16():
    from matrix_orthogonalising_optimizer_muon_amd import mixers as X
    torch.manual_seed(0)
    built = X.DecayAttention(64, 4, 16, kv_heads=2, device="cuda")
    cast = X.DecayAttention(64, 4, 16, kv_heads=2, device="cuda", dtype=torch.float32).bfloat16()
    for p, q in zip(cast.parameters(), built.parameters()):
        p.data.copy_(q)
    x = torch.randn(2, 70, 64, device="cuda").bfloat16()
    with torch.no_grad():
        (y, s), (z, t) = cast(x, final=True), built(x, final=True)
        assert torch.equal(y, z) and torch.equal(s, t)
        assert torch.equal(cast.step(x[:, 0], s), built.step(x[:, 0], t)) and torch.equal(s, t)
