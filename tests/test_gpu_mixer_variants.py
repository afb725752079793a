"""Every kernel of linear attention's walk against the float64 oracle, element by element, with the bounds of what
the kernels round: scores and the state's copy to 16 bits, results once."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import mixer as om  # noqa: E402
from tests.gpu_util import TORCH_DT, to_np  # noqa: E402
from tests.mixer_cases import CASES  # noqa: E402

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def X():
    from matrix_orthogonalising_optimizer_muon_amd import mixers
    return mixers


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", CASES)
def test_against_the_oracle(X, size, dtype):
    B, T, H, kv, D, E = size
    rng = np.random.default_rng([9, *size])
    new = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).cuda()  # noqa: E731
    q, k, v, do = (new(B, T, h, d).to(TORCH_DT[dtype]) for h, d in ((H, D), (kv, D), (kv, E), (H, E)))
    g = torch.from_numpy(-np.geomspace(1.0, 3e-4, H).astype(np.float32)).cuda()
    s, df = new(B, H, D, E) * 4.0, new(B, H, D, E) * 4.0
    lens = torch.tensor([T - (7 * b) % 130 for b in range(B)], dtype=torch.int32, device="cuda")
    f, h = float(np.float32(1.0 / np.sqrt(D))), HALF_STEP[dtype]
    kw = dict(state=s, lengths=lens)
    o, last = X.linear_attention_forward(q, k, v, g, **kw, final=True)
    dq, dk, dv, ds = X.linear_attention_backward(do, q, k, v, g, **kw, d_final=df, need_dstate=True)
    group = H // kv
    for b, j in {(0, 0), (B // 2, kv // 2), (B - 1, kv - 1)}:
        n, at = int(lens[b]), slice(j * group, (j + 1) * group)
        mine = lambda t, heads: to_np(t[b:b + 1, :n, heads])  # noqa: E731
        a = (mine(q, at), mine(k, slice(j, j + 1)), mine(v, slice(j, j + 1)), to_np(g[at]), f)
        ndo, ns, ndf = mine(do, at), to_np(s[b:b + 1, at]), to_np(df[b:b + 1, at])
        # two parts of 8 bits: wrong by at most 2^-17 of itself, and as much again for the product of two such
        kw = dict(state=ns, operands=2.0 ** -16)
        want = (*om.forward(*a, ns), *om.backward(ndo, *a, ns, None, ndf))
        limit = (*om.bounds(*a, h, **kw), *om.bounds(*a, h, do=ndo, d_final=ndf, **kw))
        got = (mine(o, at), to_np(last[b:b + 1, at]), mine(dq, at), mine(dk, slice(j, j + 1)), mine(dv, slice(j, j + 1)),
               to_np(ds[b:b + 1, at]))
        for x, r, e, name in zip(got, want, limit, ("o", "states", "dq", "dk", "dv", "dstate")):
            bad = ~(np.abs(x - r) <= e)
            assert not bad.any(), (name, b, j, int(bad.sum()), np.argwhere(bad)[:3].tolist(), x[bad][:3], r[bad][:3], e[bad][:3])
    for b in range(B):
        assert all(bool((t[b, int(lens[b]):] == 0).all()) for t in (o, dq, dk, dv))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(1, 1, 2, 1, 16, 16), (3, 150, 4, 2, 64, 40), (1, 1500, 4, 2, 126, 127), (1, 1500, 4, 2, 128, 128), (16, 330, 4, 4, 250, 256)])
def test_the_states_gradient_without_that_of_v(X, size, dtype):
    """Made by a walk without outputs: the same sums."""
    B, T, H, kv, D, E = size
    q, k, v, do = (torch.randn(B, T, h, d, device="cuda").to(TORCH_DT[dtype]) for h, d in ((H, D), (kv, D), (kv, E), (H, E)))
    g = torch.linspace(-0.5, -0.001, H, device="cuda")
    s, df = torch.randn(B, H, D, E, device="cuda"), torch.randn(B, H, D, E, device="cuda")
    lens = torch.tensor([max(T - 70 * b, 0) for b in range(B)], dtype=torch.int32, device="cuda")
    a, ns = [to_np(t) for t in (q, k, v, g)], lens.tolist()
    f = float(np.float32(1.0 / np.sqrt(D)))
    want = om.backward(to_np(do), *a, f, to_np(s), ns, to_np(df))[3]
    limit = om.bounds(*a, f, HALF_STEP[dtype], to_np(s), ns, to_np(do), to_np(df))[3]
    for need in ((False, False, False), (True, False, False), (False, True, False), (True, True, False)):
        got = X.linear_attention_backward(do, q, k, v, g, state=s, lengths=lens, d_final=df, need=need, need_dstate=True)
        assert np.all(np.abs(to_np(got[3]) - want) <= limit), need


@pytest.mark.parametrize("apart", [1 << 22, (1 << 22) + 8])
def test_rows_as_far_apart_as_direct_loads_go(X, apart):
    """Chunks that span 2^29 bytes, the most that goes through buffers, and a little more, which does not."""
    if torch.cuda.mem_get_info()[0] < (8 << 30):
        pytest.skip("needs 8 GB")
    T, D = 100, 40
    q, k, v, do = (torch.randn(1, T, 1, D, device="cuda").bfloat16() for _ in range(4))
    g, lens = torch.tensor([-0.05], device="cuda"), torch.tensor([T - 7], dtype=torch.int32, device="cuda")
    far = torch.full(((T - 1) * apart + D,), float("nan"), dtype=torch.bfloat16, device="cuda").as_strided((1, T, 1, D), (0, apart, 0, 1))

    def results(k):
        o, s = X.linear_attention_forward(q, k, v, g, lengths=lens, final=True)
        return (o, s, *X.linear_attention_backward(do, q, k, v, g, lengths=lens, need_dstate=True))
    want = results(k)
    far[:, :T - 7].copy_(k[:, :T - 7])
    assert all(torch.equal(a, b) for a, b in zip(results(far), want))
