"""What the training operators write into given tensors, torch's automatic differentiation sees:
a node that saved such a tensor refuses its backward instead of reading what was written."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    from matrix_orthogonalising_optimizer_muon_amd import layers, losses
    return layers, losses


def test_losses_in_place_raise_the_version(mods):
    S = mods[1]
    n, V = 6, 500
    t = torch.randint(0, V, (n,), device="cuda")
    old, adv = torch.full((n,), -6.0, device="cuda"), torch.randn(n, device="cuda")
    top, ids = torch.randn(n, 4, device="cuda"), torch.randint(0, V, (n, 4), device="cuda")
    for call in (lambda z: S.policy_loss(z, t, old, adv, out=z), lambda z: S.distill_loss(z, top, ids, out=z)):
        w = torch.randn(n, V, device="cuda", requires_grad=True)
        z = w * 2.0
        square = (z * z).sum()          # saves z
        before = z._version
        with torch.no_grad():
            call(z)
        assert z._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            square.backward()
        # a column range of a wider buffer: the buffer's version
        wide = torch.randn(n, V + 12, device="cuda")
        before = wide._version
        call(wide[:, 5:V + 5])
        assert wide._version > before
    # nothing given, nothing raised: the logits stay what they were
    z = torch.randn(n, V, device="cuda")
    for call in (lambda: S.policy_loss(z, t, old, adv), lambda: S.distill_loss(z, top, ids)):
        before = z._version
        call()
        assert z._version == before
    with torch.inference_mode():        # tensors without a version
        z = torch.randn(n, V, device="cuda")
        S.policy_loss(z, t, old, adv, out=z)


def test_given_gradient_buffers_raise_their_version(mods):
    L = mods[0]
    make = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    x, wg, wu, wd, dy = make(40, 16), make(24, 16), make(24, 16), make(16, 24), make(40, 16)
    _, saved = L.ffn_forward(x, wg, wu, wd, save=True)
    G = [torch.zeros_like(w) for w in (wg, wu, wd)]
    scale = torch.ones((), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    norm = (G[0] * scale).sum()         # saves G[0]
    for accumulate in (False, True):
        before = [g._version for g in G]
        L.ffn_backward(dy, x, wg, wu, wd, saved, grads=G, accumulate=accumulate)
        assert all(g._version > b for g, b in zip(G, before))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        norm.backward()
    before = G[1]._version
    L.ffn_backward(dy, x, wg, wu, wd, saved, grads=(G[0], None, None))
    assert G[1]._version == before
