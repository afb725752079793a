"""The training operators together with the updates, as a program uses them: loss with its
gradient, feed-forward backward into the persistent gradient buffers, Muon and AdamW steps."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from oracle import ffn as of  # noqa: E402
from oracle import losses as ol  # noqa: E402
from oracle import muon as om  # noqa: E402
from tests.gpu_util import rel, to_np  # noqa: E402


def rounded(rng, *shape, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).cuda().bfloat16()


def test_loss_block_update_in_sequence():
    """head(ffn(x)) -> policy loss with gradient -> block backward accumulated over two
    micro-batches into G -> one Muon step; each stage against the oracle on the stage's own inputs."""
    from matrix_orthogonalising_optimizer_muon_amd import layers, losses
    from matrix_orthogonalising_optimizer_muon_amd.optimizer import MuonUpdate
    rng = np.random.default_rng(11)
    T, D, F, V = 48, 96, 256, 500
    wg, wu, wd = rounded(rng, F, D, scale=0.1), rounded(rng, F, D, scale=0.1), rounded(rng, D, F, scale=0.06)
    head = rounded(rng, V, D, scale=0.1)
    masters = [w.float() for w in (wg, wu, wd)]
    G = [torch.zeros_like(w) for w in (wg, wu, wd)]
    M = [torch.zeros_like(w) for w in (wg, wu, wd)]
    update = MuonUpdate(list(zip(masters, G, M)), lr=0.02)
    ref = [np.zeros(w.shape) for w in (wg, wu, wd)]
    tol = [np.zeros(w.shape) for w in (wg, wu, wd)]
    before = [to_np(w) for w in masters]
    for step in range(2):
        x = rounded(rng, T, D)
        y, saved = layers.ffn_forward(x, wg, wu, wd, save=True)
        logits = y.float() @ head.float().T
        t = torch.from_numpy(rng.integers(0, V, T)).cuda()
        old = torch.log_softmax(logits, 1).gather(1, t[:, None])[:, 0] - 0.05
        adv = torch.from_numpy(rng.standard_normal(T).astype(np.float32)).cuda()
        loss, logp, dlogits = losses.policy_loss(logits, t, old.contiguous(), adv)
        want = ol.policy(to_np(logits), t.cpu().numpy(), to_np(old), to_np(adv), clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                         temperature=1.0, half_step=2.0 ** -24)
        assert np.all(np.abs(to_np(dlogits) - want["grad"]) <= want["err_grad"])
        dy = (dlogits @ head.float()).bfloat16()
        layers.ffn_backward(dy, x, wg, wu, wd, saved, grads=G, accumulate=step > 0)
        a = [to_np(v) for v in (x, wg, wu, wd)]
        for k, (r, b) in enumerate(zip(of.backward(to_np(dy), *a, "silu")[1:], of.bounds(*a, "silu", 2.0 ** -8, to_np(dy))[1:])):
            ref[k] += r
            tol[k] += b + 2.0 ** -8 * np.abs(ref[k])
    for k in range(3):
        assert np.all(np.abs(to_np(G[k]) - ref[k]) <= 1.02 * tol[k]), k
    g_used = [to_np(g) for g in G]
    update.step()
    torch.cuda.synchronize()
    for k in range(3):
        mode = "gram" if max(G[k].shape) / min(G[k].shape) > 1.5 else "plain"
        _, _, O = om.muon_step(before[k], g_used[k], np.zeros(G[k].shape), mode=mode)
        assert rel((before[k] - to_np(masters[k])) / 0.02, O) <= 2e-2
    update.close()


def test_module_under_the_torch_optimizer():
    """GatedFeedForward and a head under MuonWithAdamW: the block's matrices take the Muon
    update, the head AdamW; gradients equal the explicit calls'."""
    from matrix_orthogonalising_optimizer_muon_amd import layers, losses
    from matrix_orthogonalising_optimizer_muon_amd.optimizer import MuonWithAdamW
    torch.manual_seed(0)
    T, D, F, V, K = 64, 64, 192, 300, 8
    block = layers.GatedFeedForward(D, F, device="cuda")
    head = torch.nn.Linear(D, V, bias=False, device="cuda", dtype=torch.bfloat16)
    params = [(f"block.{n}", p) for n, p in block.named_parameters()] + [("lm_head.weight", head.weight)]
    opt = MuonWithAdamW(params, lr=0.02, adamw_lr=1e-3)
    assert len(opt.muon_parameters()) == 3 and len(opt.adamw_parameters()) == 1
    x = torch.randn(T, D, device="cuda").bfloat16()
    top = torch.randn(T, K, device="cuda")
    ids = torch.randperm(V, device="cuda")[:K].repeat(T, 1)
    for _ in range(2):
        opt.zero_grad()
        y = block(x)
        y.retain_grad()
        z = head(y)
        losses.distill_loss_rows(z, top, ids, temperature=2.0).mean().backward()
        _, saved = layers.ffn_forward(x, block.gate, block.up, block.down, save=True)
        want = layers.ffn_backward(y.grad, x, block.gate, block.up, block.down, saved, need_dx=False)
        for p, w in zip((block.gate, block.up, block.down), want[1:]):
            assert torch.equal(p.grad, w)
        before = [p.detach().clone() for p in opt.muon_parameters()]
        opt.step()
        torch.cuda.synchronize()
        for p, b in zip(opt.muon_parameters(), before):
            assert bool(torch.isfinite(p).all()) and not torch.equal(p, b)


def test_backward_in_a_captured_graph():
    """Forward and backward of the block and a loss captured in one graph, replayed against
    eager passes."""
    from matrix_orthogonalising_optimizer_muon_amd import layers, losses
    torch.manual_seed(1)
    x = torch.randn(40, 72, device="cuda").bfloat16()
    ws = [(0.1 * torch.randn(s, device="cuda")).bfloat16().requires_grad_(True) for s in ((136, 72), (136, 72), (72, 136))]
    top, ids = torch.randn(40, 5, device="cuda"), torch.randint(0, 72, (40, 5), device="cuda")

    def step():
        y = layers.gated_ffn(x, *ws)
        loss = losses.distill_loss_rows(y, top, ids)
        return (loss.detach(), *torch.autograd.grad(loss.sum(), ws))
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for k in range(3):
        x.copy_(torch.randn(40, 72, device="cuda"))
        g.replay()
        torch.randn(1 << 18, device="cuda").add_(1.0)
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), k
