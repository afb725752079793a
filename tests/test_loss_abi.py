"""C-ABI checks of the losses beyond test_train_abi.py, on a host-only context."""

import pytest

B = pytest.importorskip("matrix_orthogonalising_optimizer_muon_amd.binding")
FAKE = 0x100000  # never dereferenced: host-only contexts launch nothing


@pytest.fixture(scope="module")
def hctx():
    ctx = B.muon_init(-1)
    yield ctx
    B.muon_destroy(ctx)


def logits(**kw):
    d = dict(logits=FAKE, dlogits=FAKE * 2, weights=None, grad_rows=None, loss=FAKE, lse=FAKE, ld=50, ld_d=50, rows=3,
             vocab=50, temperature=1.0, dtype=B.MUON_BF16, lse_given=0)
    d.update(kw)
    return B.muon_logits(**d)


def both(ctx, l):
    p = B.muon_policy(targets=FAKE, old_logp=FAKE, advantages=FAKE, ref_logp=FAKE, logp=FAKE, clip_low=0.2, clip_high=0.2,
                      kl_coef=0.1)
    t = B.muon_distill(top_logits=FAKE, top_ids=FAKE, top_lse=None, ld_top=4, ld_ids=4, top=4, top_dtype=B.MUON_F32,
                       id_dtype=B.MUON_I64)
    return B.muon_policy_loss(ctx, l, p, None, 0, None), B.muon_distill_loss(ctx, l, t, None, 0, None)


def test_pairs_in_place_of_one_normaliser(hctx):
    ok, bad = (B.MUON_ERR_DEVICE,) * 2, (B.MUON_ERR_ARG,) * 2
    for kw, want in [(dict(lse_pairs=1), ok), (dict(lse_pairs=1, lse_given=1), ok), (dict(lse_pairs=1, lse=None), ok),
                     (dict(lse_pairs=1, lse_given=1, lse=None), bad), (dict(lse_pairs=2), bad), (dict(lse_pairs=-1), bad)]:
        assert both(hctx, logits(**kw)) == want, kw


def test_workspace_size_of_sizes_that_the_losses_refuse(hctx):
    """The size query has the losses' own limits: past them it would compute with what overflows."""
    import ctypes
    n = ctypes.c_size_t()
    size = lambda **kw: B._lib.muon_loss_workspace_size(hctx, logits(**kw), 0, n)  # noqa: E731
    assert size(rows=(1 << 24) - 1) == B.MUON_OK and size(vocab=1 << 28) == B.MUON_OK and size(rows=0) == B.MUON_OK
    for bad in [dict(rows=1 << 24), dict(rows=1 << 62), dict(vocab=(1 << 28) + 1), dict(vocab=1 << 62), dict(lse_given=2)]:
        assert size(**bad) == B.MUON_ERR_ARG, bad
    # it depends on the sizes alone: pointers and strides may still be missing
    assert size(logits=None, dlogits=None, ld=0, ld_d=0, lse=None) == B.MUON_OK
