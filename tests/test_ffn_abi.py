"""C-ABI checks of the feed-forward block beyond test_train_abi.py, on a host-only context."""

import pytest

B = pytest.importorskip("matrix_orthogonalising_optimizer_muon_amd.binding")
FAKE = 0x100000  # never dereferenced: host-only contexts launch nothing
T, D, F = 10, 40, 72


@pytest.fixture(scope="module")
def hctx():
    ctx = B.muon_init(-1)
    yield ctx
    B.muon_destroy(ctx)


def block(**kw):
    d = dict(x=FAKE, w_gate=FAKE, w_up=FAKE, w_down=FAKE, ld_x=D, ld_gate=D, ld_up=D, ld_down=F, tokens=T, dim=D, hidden=F,
             dtype=B.MUON_BF16, activation=0)
    d.update(kw)
    return B.muon_ffn(**d)


def grads(*wanted, **kw):
    d = dict(dy=FAKE, saved=FAKE, ld_dy=D, ld_dx=D, ld_g_gate=D, ld_g_up=D, ld_g_down=F, g_dtype=B.MUON_BF16, accumulate=0)
    d.update({w: FAKE for w in wanted}, **kw)
    return B.muon_ffn_grads(**d)


def test_backward_copies_only_what_a_wanted_gradient_reads(hctx):
    """Rows off 16 bytes are copied into the workspace: w_gate and w_up for dx alone, x for g_gate and
    g_up alone, dy and w_down always."""
    need = lambda f, g: B.muon_ffn_workspace_size(hctx, f, g)[0]  # noqa: E731
    off_weights, off_x = block(ld_gate=D + 1, ld_up=D + 1), block(ld_x=D + 1)
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    for wanted in [("dx",), ("g_gate",), ("g_up",), ("g_down",), ("g_gate", "g_up", "g_down"), ("dx", "g_down"),
                   ("dx", "g_gate", "g_up", "g_down")]:
        g = grads(*wanted)
        base = need(block(), g)
        assert need(off_weights, g) - base == (2 * up(F * D * 2) if "dx" in wanted else 0), wanted
        assert need(off_x, g) - base == (up(T * D * 2) if {"g_gate", "g_up"} & set(wanted) else 0), wanted
        assert need(block(ld_down=F + 1), g) - base == up(D * F * 2), wanted
        assert need(block(), grads(*wanted, ld_dy=D + 1)) - base == up(T * D * 2), wanted
        # two strides, both aligned: one of the weights is copied, for dx alone
        assert (need(block(ld_gate=D + 8), g) > base) == ("dx" in wanted), wanted
        for f in (off_weights, off_x):
            n = need(f, g)
            assert B.muon_ffn_backward(hctx, f, g, FAKE, n, None) == B.MUON_ERR_DEVICE
            assert B.muon_ffn_backward(hctx, f, g, FAKE, n - 1, None) == B.MUON_ERR_WORKSPACE
