"""Dropout from a counter (muon_dropout): the mask against the integers of the oracle, the values
within one rounding."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import dropout as od  # noqa: E402
from tests.gpu_util import TORCH_DT, to_np  # noqa: E402

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SEED, OFFSET = 0x9E3779B97F4A7C15, (1 << 40) + 12345


@pytest.fixture(scope="module")
def R():
    from matrix_orthogonalising_optimizer_muon_amd import dropout
    return dropout


def draw(dtype, *shape, seed=0, scale=1.0):
    rng = np.random.default_rng([seed, *shape])
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).cuda().to(TORCH_DT[dtype])


def check(got, x, p, seed, offset, residual, dtype):
    want = od.dropout(to_np(x), p, seed, offset, None if residual is None else to_np(residual))
    size = od.dropout(np.abs(to_np(x)), p, seed, offset)     # the factor and the product: two roundings in fp32
    assert np.all(np.abs(to_np(got) - want) <= 1.01 * HALF_STEP[dtype] * np.abs(want) + 3 * 2.0 ** -24 * size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (1, 1), (5, 3), (3, 8), (2, 1023), (1, 8193), (3, 5, 7), (130, 65), (9, 2048)])
def test_parity(R, shape, dtype):
    x, r = draw(dtype, *shape), draw(dtype, *shape, seed=1, scale=4.0)
    for p, seed, offset in ((0.1, SEED, OFFSET), (0.5, -3, 0), (0.37, 0, (1 << 64) - 1)):
        for res in (None, r):
            check(R.dropout_forward(x, p, seed, offset, residual=res), x, p, seed % (1 << 64), offset, res, dtype)
        check(R.dropout_backward(x, p, seed, offset), x, p, seed % (1 << 64), offset, None, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_edges_of_p(R, dtype):
    x, r = draw(dtype, 40, 100), draw(dtype, 40, 100, seed=1)
    assert torch.equal(R.dropout_forward(x, 0.0, 1), x) and torch.equal(R.dropout_forward(x, 2.0 ** -18, 1), x)
    assert bool((R.dropout_forward(x, 1.0, 1) == 0).all()) and torch.equal(R.dropout_forward(x, 1.0, 1, residual=r), r)
    for p in (2.0 ** -17, 2.0 ** -16, 1 - 2.0 ** -16, 0.99999):
        check(R.dropout_forward(x, p, SEED), x, p, SEED, 0, None, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_is_dropped_is_not_used(R, dtype):
    x = draw(dtype, 64, 33)
    keep = torch.from_numpy((od.numbers(x.numel(), 5, 6) >= od.threshold(0.5)).reshape(64, 33)).cuda()
    dirty = torch.where(keep, x, torch.tensor(float("nan"), dtype=x.dtype, device="cuda"))
    assert torch.equal(R.dropout_forward(dirty, 0.5, 5, 6), R.dropout_forward(x, 0.5, 5, 6))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off,extra", [(0, 1), (1, 0), (8, 24), (3, 5)])
@pytest.mark.parametrize("cols", [5, 64, 203])
def test_strided(R, dtype, off, extra, cols):
    """The mask goes by an element's number, not by where it lies; nothing around is touched."""
    x, r = draw(dtype, 30, cols), draw(dtype, 30, cols, seed=1)
    want = R.dropout_forward(x, 0.3, 11, residual=r)
    wide = lambda: torch.full((32, off + cols + extra), float("nan"), dtype=x.dtype, device="cuda")  # noqa: E731
    a, b, o = wide(), wide(), wide()
    va, vb, vo = (t[1:-1, off:off + cols] for t in (a, b, o))
    va.copy_(x)
    vb.copy_(r)
    assert torch.equal(R.dropout_forward(va, 0.3, 11, residual=vb), want)
    before = o._version
    assert R.dropout_forward(x, 0.3, 11, residual=vb, out=vo) is vo and o._version > before
    assert torch.equal(vo, want) and int(torch.isnan(o).sum()) == o.numel() - vo.numel()
    R.dropout_forward(x, 0.3, 11, residual=vb, out=vb)          # in place of the residual
    assert torch.equal(vb, want)
    R.dropout_forward(va, 0.3, 11, out=va)                      # in place of x
    assert torch.equal(va, R.dropout_forward(x, 0.3, 11)) and int(torch.isnan(a).sum()) == a.numel() - va.numel()


def test_a_tensor_for_the_seed(R):
    x = draw("bf16", 50, 72)
    c = torch.tensor([SEED - (1 << 64), 9], dtype=torch.int64, device="cuda")
    assert torch.equal(R.dropout_forward(x, 0.2, c), R.dropout_forward(x, 0.2, SEED, 9))
    leaf = x.clone().requires_grad_(True)
    y = R.dropout(leaf, 0.2, c)
    c[1] += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_automatic_differentiation(R):
    x, r = draw("f32", 6, 5, 40).requires_grad_(True), draw("f32", 6, 5, 40, seed=2).requires_grad_(True)
    up = draw("f32", 6, 5, 40, seed=3)
    y = R.dropout(x, 0.4, 77, 5, residual=r)
    gx, gr = torch.autograd.grad((y * up).sum(), (x, r))
    assert torch.equal(gr, up) and torch.equal(gx, R.dropout_forward(up, 0.4, 77, 5))
    gx = torch.autograd.grad(R.dropout(x, 0.4, 77, 5).sum(), x)[0]    # an expanded gradient
    assert torch.equal(gx, R.dropout_forward(torch.ones_like(up), 0.4, 77, 5))
    # linear in x: the difference of two outputs is the gradient's product, but for fp32's roundings
    d = R.dropout_forward(x.detach() + up, 0.4, 77, 5).double() - R.dropout_forward(x.detach(), 0.4, 77, 5).double()
    assert float((d - gx.double() * up.double()).abs().max()) <= 8 * 2.0 ** -24 * float(x.detach().abs().max() + up.abs().max()) * 2


def test_module_counts_its_calls(R):
    m = R.Dropout(0.3, seed=-5, device="cuda")
    x, r = draw("bf16", 20, 64), draw("bf16", 20, 64, seed=1)
    for n in range(3):
        assert torch.equal(m(x, r), R.dropout_forward(x, 0.3, -5, n, residual=r))
    m.eval()
    assert torch.equal(m(x), x) and torch.equal(m(x, r), x + r) and m.counter.tolist() == [-5, 3]


def test_captured_and_replayed(R):
    """Each replay draws the next mask, as eager calls do."""
    m, e = R.Dropout(0.25, seed=3, device="cuda"), R.Dropout(0.25, seed=3, device="cuda")
    x = draw("bf16", 33, 100).requires_grad_(True)

    def step(mod):
        y = mod(x)
        return y.detach(), torch.autograd.grad(y.float().square().sum(), x)[0]
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step(m)
    torch.cuda.current_stream().wait_stream(warm)
    step(e)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step(m)
    for k in range(4):
        g.replay()
        torch.randn(1 << 18, device="cuda").add_(1.0)
        want = step(e)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), k


def test_large(R):
    """More than 2^32 bytes: a far part against the same elements alone."""
    if torch.cuda.mem_get_info()[0] < (24 << 30):
        pytest.skip("needs 24 GB")
    n = (1 << 31) + 8 * 1001 + 3
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = R.dropout_forward(x, 0.5, 9, 4)
    first = n - 4003
    b0 = first // 8
    words = np.array([od.philox((b & od.M32, b >> 32, 4, 0), (9, 0)) for b in range(b0, (n + 7) // 8)])
    want = np.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[first - 8 * b0:][:4003] >= 32768
    assert np.array_equal(y[first:].float().cpu().numpy() != 0, want)
    # kept: 2^31 draws of 1/2; six deviations
    kept = float((y != 0).sum(dtype=torch.float64))
    assert abs(kept / n - 0.5) <= 6 * 0.5 / np.sqrt(n)


def test_refusals(R):
    x = torch.randn(6, 8, device="cuda")
    for bad, kind in [(lambda: R.dropout_forward(x.half(), 0.1, 1), TypeError), (lambda: R.dropout_forward(x.cpu(), 0.1, 1), ValueError),
                      (lambda: R.dropout_forward(x, -0.1, 1), ValueError), (lambda: R.dropout_forward(x, 1.1, 1), ValueError),
                      (lambda: R.dropout_forward(x, float("nan"), 1), ValueError), (lambda: R.dropout_forward(x, 0.1, 1.5), TypeError),
                      (lambda: R.dropout_forward(x, 0.1, 1 << 64), ValueError), (lambda: R.dropout_forward(x, 0.1, 1, -(1 << 63) - 1), ValueError),
                      (lambda: R.dropout_forward(x, 0.1, 1, residual=x[:5]), ValueError),
                      (lambda: R.dropout_forward(x, 0.1, 1, residual=x.bfloat16()), TypeError),
                      (lambda: R.dropout_forward(x, 0.1, 1, residual=x.cpu()), ValueError),
                      (lambda: R.dropout_forward(x.t(), 0.1, 1), ValueError),
                      (lambda: R.dropout_forward(x, 0.1, torch.zeros(2, device="cuda")), TypeError),
                      (lambda: R.dropout_forward(x, 0.1, torch.zeros(3, dtype=torch.int64, device="cuda")), ValueError),
                      (lambda: R.dropout_forward(x, 0.1, torch.zeros(2, dtype=torch.int64, device="cuda"), 1), ValueError),
                      (lambda: R.dropout_forward(x[:5], 0.1, 1, out=x[1:]), Exception),
                      (lambda: R.Dropout(1.5), ValueError)]:
        with pytest.raises(kind):
            bad()
    assert R.dropout_forward(x[:0], 0.1, 1).shape == (0, 8)
