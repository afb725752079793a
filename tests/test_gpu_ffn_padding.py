"""Feed-forward blocks whose last tile lies in the padding of the hidden size while the last slice
of the summed size has one row left, with rows that are read in place."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import ffn as of  # noqa: E402
from tests.gpu_util import to_np  # noqa: E402


@pytest.mark.parametrize("dtype,T,D,F", [(torch.bfloat16, 16, 65, 72), (torch.bfloat16, 1, 193, 136),
                                         (torch.bfloat16, 16, 3585, 8136), (torch.float32, 5, 33, 68),
                                         (torch.float32, 40, 97, 132)])
def test_ffn_tiles_in_the_padding(dtype, T, D, F):
    from matrix_orthogonalising_optimizer_muon_amd import layers as L
    gen = torch.Generator("cuda").manual_seed(6)
    make = lambda r, c, s: (s * torch.randn(r, c, generator=gen, device="cuda")).to(dtype)  # noqa: E731
    x, wg, wu = make(T, D, 1.0), make(F, D, D ** -0.5), make(F, D, D ** -0.5)
    wd, dy = make(D, F, F ** -0.5), make(T, D, 0.5)
    y, saved = L.ffn_forward(x, wg, wu, wd, save=True)
    got = (y, *L.ffn_backward(dy, x, wg, wu, wd, saved))
    ops, e = [to_np(t) for t in (x, wg, wu, wd)], torch.finfo(dtype).eps / 2
    want = (of.forward(*ops, "silu"), *of.backward(to_np(dy), *ops, "silu"))
    bound = (of.bounds(*ops, "silu", e), *of.bounds(*ops, "silu", e, to_np(dy)))
    for a, r, b in zip(got, want, bound):
        assert np.all(np.abs(to_np(a) - r) <= b)
