"""The gated feed-forward block (muon_ffn_forward, muon_ffn_backward) against the float64
oracle, element by element, within the errors oracle.ffn.bounds derives from the storage
type's half step and fp32 sums."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import ffn as of  # noqa: E402
from tests.gpu_util import TORCH_DT, to_np  # noqa: E402

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def L():
    from matrix_orthogonalising_optimizer_muon_amd import layers
    return layers


def block(T, D, F, dtype, seed=0):
    """x, w_gate, w_up, w_down, dy on the GPU: values of the storage type."""
    rng = np.random.default_rng([seed, T, D, F])
    def make(r, c, scale):
        return torch.from_numpy((scale * rng.standard_normal((r, c))).astype(np.float32)).cuda().to(TORCH_DT[dtype])
    return (make(T, D, 1.0), make(F, D, 2.0 / np.sqrt(D)), make(F, D, 1.0 / np.sqrt(D)), make(D, F, 1.0 / np.sqrt(F)),
            make(T, D, 0.5))


def inside(got, ref, bound, what):
    err = np.abs(to_np(got) - ref)
    bad = ~(err <= bound + 1e-37)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.max(err / (bound + 1e-37))))


def check(L, ops, act, dtype, g_dtype=None, old=None):
    x, wg, wu, wd, dy = ops
    a = [to_np(t) for t in (x, wg, wu, wd)]
    y, saved = L.ffn_forward(x, wg, wu, wd, activation=act, save=True)
    e = HALF_STEP[dtype]
    inside(y, of.forward(*a, act), of.bounds(*a, act, e), "y")
    y2, none = L.ffn_forward(x, wg, wu, wd, activation=act)
    assert none is None and torch.equal(y, y2)
    gd = g_dtype or dtype
    grads = None
    if g_dtype or old is not None:
        grads = tuple(torch.full(w.shape, 0.0 if old is None else old, dtype=TORCH_DT[gd], device="cuda") for w in (wg, wu, wd))
    out = L.ffn_backward(dy, x, wg, wu, wd, saved, activation=act, grads=grads, accumulate=old is not None)
    ref = of.backward(to_np(dy), *a, act)
    bound = of.bounds(*a, act, e, to_np(dy), HALF_STEP[gd])
    for k, name in enumerate(("dx", "g_gate", "g_up", "g_down")):
        r, b = ref[k], bound[k]
        if old is not None and k:   # the sum is rounded, not the gradient alone
            b = b + (HALF_STEP[gd] + 2.0 ** -23) * (np.abs(r + old) + b)
            r = r + old
        inside(out[k], r, b, name)
    return y, out


SIZES = [(1, 64, 64), (1, 8, 1), (2, 1, 1), (3, 7, 5), (16, 64, 128), (17, 72, 200), (33, 413, 111), (63, 65, 63),
         (64, 128, 64), (65, 129, 257), (100, 256, 1024), (129, 200, 520), (200, 1000, 96), (257, 640, 320),
         (300, 40, 1000), (513, 96, 72)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,F", SIZES)
def test_ffn_parity(L, T, D, F, dtype, act):
    check(L, block(T, D, F, dtype), act, dtype)


@pytest.mark.parametrize("T,D,F", [(2300, 1600, 2304), (2049, 2051, 1283)])
def test_ffn_parity_large_tiles(L, T, D, F):
    """Enough tiles for the 256 x 256 kernels, aligned and ragged."""
    check(L, block(T, D, F, "bf16"), "silu", "bf16")


@pytest.mark.parametrize("T,D,F", [(8, 64, 20000), (40, 64, 9001), (20000, 64, 64), (9001, 72, 80)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ffn_parity_long_sums(L, T, D, F, dtype):
    """Few output tiles and long sums: the split of K."""
    check(L, block(T, D, F, dtype), "silu", dtype)


@pytest.mark.parametrize("dtype,g_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,D,F", [(70, 72, 136), (33, 41, 59), (9001, 64, 64)])
def test_ffn_accumulates_into_given_buffers(L, T, D, F, dtype, g_dtype):
    check(L, block(T, D, F, dtype), "silu", dtype, g_dtype=g_dtype)
    check(L, block(T, D, F, dtype), "silu", dtype, g_dtype=g_dtype, old=0.25)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off,extra", [(0, 8), (8, 16), (1, 3), (3, 0)])
def test_ffn_strided_operands(L, dtype, off, extra):
    """Operands inside wider buffers that hold NaN around them: nothing outside is read into a
    result, nothing outside an output is written."""
    T, D, F = 45, 90, 150
    ops = block(T, D, F, dtype)
    y0, out0 = check(L, ops, "silu", dtype)

    def inside_of(t):
        wide = torch.full((t.shape[0] + 2, t.shape[1] + off + extra), float("nan"), dtype=t.dtype, device="cuda")
        view = wide[1:-1, off:off + t.shape[1]]
        view.copy_(t)
        return wide, view
    pairs = [inside_of(t) for t in ops]
    x, wg, wu, wd, dy = (v for _, v in pairs)
    y, saved = L.ffn_forward(x, wg, wu, wd, save=True)
    outs = [inside_of(w) for w in (wg, wu, wd)]
    got = L.ffn_backward(dy, x, wg, wu, wd, saved, grads=tuple(v for _, v in outs))
    assert torch.equal(y, y0)
    for a, b in zip(got, out0):
        assert torch.equal(a, b)
    for wide, view in outs:   # the frame around each output still holds NaN
        frame = torch.isnan(wide)
        frame[1:-1, off:off + view.shape[1]] = True
        assert bool(frame.all())


@pytest.mark.parametrize("gate_extra,up_extra", [(0, 8), (24, 0), (8, 3), (3, 5)])
def test_ffn_weights_of_different_strides(L, gate_extra, up_extra):
    """w_gate and w_up with row strides of their own, and gradient buffers likewise."""
    T, D, F = 37, 72, 140
    ops = list(block(T, D, F, "bf16"))
    y0, out0 = check(L, ops, "silu", "bf16")
    for k, extra in ((1, gate_extra), (2, up_extra)):
        wide = torch.full((F, D + extra), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :D] = ops[k]
        ops[k] = wide[:, :D]
    x, wg, wu, wd, dy = ops
    y, saved = L.ffn_forward(x, wg, wu, wd, save=True)
    grads = (torch.empty(F, D + up_extra, dtype=torch.bfloat16, device="cuda")[:, :D],
             torch.empty(F, D + gate_extra, dtype=torch.bfloat16, device="cuda")[:, :D], torch.empty_like(wd))
    got = L.ffn_backward(dy, x, wg, wu, wd, saved, grads=grads)
    assert torch.equal(y, y0) and all(torch.equal(a, b) for a, b in zip(got, out0))


def test_ffn_nan_stays_in_its_row(L):
    """A NaN or infinity in one token reaches that token's results and the weight gradients' columns
    only through the formulas: other rows of y and dx are what they were."""
    T, D, F = 40, 70, 90
    x, wg, wu, wd, dy = block(T, D, F, "bf16")
    y0, s0 = L.ffn_forward(x, wg, wu, wd, save=True)
    dx0 = L.ffn_backward(dy, x, wg, wu, wd, s0)[0]
    x = x.clone()
    x[7, 69] = float("nan")
    x[39, 0] = float("inf")
    y, s = L.ffn_forward(x, wg, wu, wd, save=True)
    dx = L.ffn_backward(dy, x, wg, wu, wd, s)[0]
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[7, 39]] = False
    assert torch.equal(y[keep], y0[keep]) and torch.equal(dx[keep], dx0[keep])
    assert bool(torch.isnan(y[7]).all()) and bool(torch.isnan(dx[7]).all())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_ffn_gates_whose_square_overflows(L, act):
    """|g| = 1e25: act(g) is g or 0 and its slope 1 or 0 exactly. One hidden column of two (g u =
    1e25 u or 0), small u and down weights, so that every value is a power-of-ten product of few factors."""
    x = torch.tensor([[1.0, 0.0], [-1.0, 0.0]], device="cuda")
    wg = torch.tensor([[1e25, 0.0]], device="cuda")
    wu = torch.tensor([[2.0 ** -70, 1.0]], device="cuda")
    wd = torch.tensor([[2.0 ** -3], [2.0 ** -4]], device="cuda")
    dy = torch.tensor([[1.0, 2.0], [4.0, 8.0]], device="cuda")
    y, saved = L.ffn_forward(x, wg, wu, wd, activation=act, save=True)
    dx, g_gate, g_up, g_down = L.ffn_backward(dy, x, wg, wu, wd, saved, activation=act)
    g = float(wg[0, 0])                       # every product below is by a power of two: exact
    h, dh = g * 2.0 ** -70, 2.0 ** -3 + 2.0 ** -3
    assert y.tolist() == [[h * 2.0 ** -3, h * 2.0 ** -4], [0.0, 0.0]]
    du, dg = dh * g, dh * 2.0 ** -70
    assert g_gate.tolist() == [[dg, 0.0]] and g_up.tolist() == [[du, 0.0]] and g_down.tolist() == [[h], [2 * h]]
    want = dg * g + du * 2.0 ** -70           # two equal terms: exact
    assert dx.tolist() == [[want, du], [0.0, 0.0]]


def test_ffn_grads_that_overlap_are_refused(L):
    x, wg, wu, wd, dy = block(40, 16, 24, "bf16")
    y, saved = L.ffn_forward(x, wg, wu, wd, save=True)
    both, own = torch.zeros(24, 32, device="cuda", dtype=torch.bfloat16), torch.zeros_like(wd)
    want = L.ffn_backward(dy, x, wg, wu, wd, saved)
    got = L.ffn_backward(dy, x, wg, wu, wd, saved, grads=(both[:, :16], both[:, 16:], own))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    for grads in [(both[:, :16], both[:, :16], own), (both[:, :16], both[:, 8:24], own), (wg, both[:, :16], own),
                  (both[:, :16], both[:, 16:], wd), (x[:24], both[:, :16], own)]:
        with pytest.raises(ValueError, match="overlap"):
            L.ffn_backward(dy, x, wg, wu, wd, saved, grads=grads)


def test_ffn_extreme_gates(L):
    """Gates far outside the curved range: act(g) is g or 0 and the slope 1 or 0, no NaN."""
    T, D, F = 20, 64, 64
    x, wg, wu, wd, dy = block(T, D, F, "f32")
    for act in ("silu", "gelu_tanh"):
        check(L, (x * 300.0, wg, wu, wd, dy), act, "f32")


@pytest.mark.parametrize("wanted", [(True, False, False, False), (False, True, False, False), (False, False, True, False),
                                    (False, False, False, True), (False, True, True, False)])
def test_ffn_wanted_gradients_only(L, wanted):
    x, wg, wu, wd, dy = block(50, 72, 104, "bf16")
    _, saved = L.ffn_forward(x, wg, wu, wd, save=True)
    full = L.ffn_backward(dy, x, wg, wu, wd, saved)
    grads = tuple(torch.empty_like(w) if n else None for w, n in zip((wg, wu, wd), wanted[1:]))
    got = L.ffn_backward(dy, x, wg, wu, wd, saved, grads=grads, need_dx=wanted[0])
    for a, b, n in zip(got, full, wanted):
        assert (a is None) != n and (not n or torch.equal(a, b))


def test_ffn_no_tokens(L):
    x, wg, wu, wd, dy = block(0, 24, 40, "bf16")
    y, saved = L.ffn_forward(x, wg, wu, wd, save=True)
    assert y.shape == (0, 24)
    grads = tuple(torch.full_like(w, 3.0) for w in (wg, wu, wd))
    L.ffn_backward(dy, x, wg, wu, wd, saved, grads=grads, accumulate=True)
    assert all(bool((g == 3.0).all()) for g in grads)
    out = L.ffn_backward(dy, x, wg, wu, wd, saved, grads=grads)
    assert out[0].shape == (0, 24) and all(bool((g == 0.0).all()) for g in grads)


def test_ffn_offsets_past_32_bits(L):
    """Tokens a wide stride apart: byte offsets past 2^32."""
    T, D, F, ld = 70000, 64, 64, 32768   # 4.6 GB of buffer
    x0, wg, wu, wd, dy0 = block(T, D, F, "bf16")
    wide = torch.zeros(T, ld, dtype=torch.bfloat16, device="cuda")
    wide[:, :D] = x0
    wide[:, D:2 * D] = dy0
    y0, s0 = L.ffn_forward(x0, wg, wu, wd, save=True)
    y, s = L.ffn_forward(wide[:, :D], wg, wu, wd, save=True)
    assert torch.equal(y, y0) and torch.equal(s, s0)
    a = L.ffn_backward(dy0, x0, wg, wu, wd, s0)
    b = L.ffn_backward(wide[:, D:2 * D], wide[:, :D], wg, wu, wd, s)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    rows = slice(T - 40, T)
    ops = [to_np(t) for t in (x0[rows], wg, wu, wd)]
    inside(y[rows], of.forward(*ops, "silu"), of.bounds(*ops, "silu", 2.0 ** -8), "y")


def test_ffn_autograd(L):
    """gated_ffn under torch's automatic differentiation, with leading dimensions and an
    expanded upstream gradient."""
    x, wg, wu, wd, _ = (t.requires_grad_(True) for t in block(24, 40, 56, "bf16"))
    y = L.gated_ffn(x.view(2, 12, 40), wg, wu, wd, "gelu_tanh")
    assert y.shape == (2, 12, 40)
    got = torch.autograd.grad(y.sum(), (x, wg, wu, wd))
    a = [to_np(t) for t in (x, wg, wu, wd)]
    dy = np.ones((24, 40))
    for g, r, b in zip(got, of.backward(dy, *a, "gelu_tanh"), of.bounds(*a, "gelu_tanh", 2.0 ** -8, dy)):
        inside(g, r, b, "grad")
    only = torch.autograd.grad(L.gated_ffn(x.detach(), wg, wu.detach(), wd.detach()).sum(), (wg,))
    assert only[0].shape == wg.shape


def test_ffn_same_result_every_time(L):
    x, wg, wu, wd, dy = block(300, 200, 9000, "bf16")
    y, s = L.ffn_forward(x, wg, wu, wd, save=True)
    out = L.ffn_backward(dy, x, wg, wu, wd, s)
    for _ in range(3):
        y2, s2 = L.ffn_forward(x, wg, wu, wd, save=True)
        assert torch.equal(y, y2) and torch.equal(s, s2)
        assert all(torch.equal(a, b) for a, b in zip(out, L.ffn_backward(dy, x, wg, wu, wd, s2)))


def test_ffn_streams_and_graph(L):
    """On a side stream, and captured and replayed with other eager work between the replays."""
    ops = block(90, 136, 264, "bf16")
    x, wg, wu, wd, dy = (t.clone() for t in ops)
    x0, dy0 = ops[0], ops[4]

    def step():
        y, s = L.ffn_forward(x, wg, wu, wd, save=True)
        return (y, *L.ffn_backward(dy, x, wg, wu, wd, s))
    eager = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for k in range(4):
        x.copy_(x0 * (1.0 + k))
        dy.copy_(dy0 * (1.0 - 0.25 * k))
        g.replay()
        torch.randn(1 << 20, device="cuda").mul_(2.0)
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held)), k


def test_ffn_two_calls_at_once(L):
    """Two streams of work in flight: each call has a workspace of its own."""
    a, b = block(500, 256, 512, "bf16", 1), block(480, 264, 520, "bf16", 2)
    wa, wb = L.ffn_forward(*a[:4])[0], L.ffn_forward(*b[:4])[0]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            got.append((L.ffn_forward(*a[:4])[0], wa))
        with torch.cuda.stream(s2):
            got.append((L.ffn_forward(*b[:4])[0], wb))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in got)


def test_ffn_refusals(L):
    x, wg, wu, wd, dy = block(40, 16, 24, "bf16")   # saved holds whole blocks of 32 tokens
    y, saved = L.ffn_forward(x, wg, wu, wd, save=True)
    with pytest.raises(TypeError):
        L.ffn_forward(x, wg.float(), wu, wd)
    with pytest.raises(ValueError):
        L.ffn_forward(x, wg, wu[:-1], wd)
    with pytest.raises(ValueError):
        L.ffn_forward(x, wg, wu, wd.T.contiguous())
    with pytest.raises(ValueError, match="unit column stride"):
        L.ffn_forward(x, wg, wu, wd.T.contiguous().T)
    with pytest.raises(ValueError):
        L.ffn_forward(x, wg, wu.cpu(), wd)
    with pytest.raises(ValueError):
        L.ffn_forward(x[:, :8], wg, wu, wd)
    with pytest.raises(ValueError, match="saved"):
        L.ffn_backward(dy[:5], x[:5], wg, wu, wd, saved)
    with pytest.raises(TypeError, match="saved"):
        L.ffn_backward(dy, x, wg, wu, wd, None)
    with pytest.raises(ValueError, match="accumulate"):
        L.ffn_backward(dy, x, wg, wu, wd, saved, accumulate=True)
    with pytest.raises(TypeError):
        L.ffn_backward(dy, x, wg, wu, wd, saved, grads=(wg.float(), wu.clone(), wd.clone()))
