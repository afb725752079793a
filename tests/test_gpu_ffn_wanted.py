"""The feed-forward backward for some of its gradients, with rows off 16 bytes: the operands that
are not copied are those that no wanted gradient reads."""

import itertools

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import ffn as of  # noqa: E402
from tests.gpu_util import to_np  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,D,F", [(50, 73, 101), (1, 65, 9), (33, 64, 71)])
def test_ffn_wanted_gradients_of_unaligned_rows(T, D, F, dtype):
    from matrix_orthogonalising_optimizer_muon_amd import layers as L
    gen = torch.Generator("cuda").manual_seed(4)
    make = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    x, wg, wu, wd, dy = make(T, D), make(F, D), make(F, D), make(D, F), make(T, D)
    _, saved = L.ffn_forward(x, wg, wu, wd, save=True)
    ops = [to_np(t) for t in (x, wg, wu, wd)]
    want = of.backward(to_np(dy), *ops, "silu")
    bound = of.bounds(*ops, "silu", torch.finfo(dtype).eps / 2, to_np(dy))
    for wanted in itertools.product((False, True), repeat=4):
        grads = tuple(torch.empty_like(w) if n else None for w, n in zip((wg, wu, wd), wanted[1:]))
        got = L.ffn_backward(dy, x, wg, wu, wd, saved, grads=grads, need_dx=wanted[0])
        for a, r, b, n in zip(got, want, bound, wanted):
            assert (a is None) != n
            assert not n or np.all(np.abs(to_np(a) - r) <= b)
