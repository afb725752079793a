"""Losses over vocabulary logits, each with its gradient in one call
(``muon_policy_loss``, ``muon_distill_loss``).

``policy_loss`` and ``distill_loss`` return the rows' losses and, in the same pass over the
logits, the gradient of their sum; with ``out`` it goes to a given tensor, which may be the
logits themselves. ``policy_loss_rows`` and ``distill_loss_rows`` are the same losses for
torch's automatic differentiation (the forward keeps each row's maximum and sum, the backward
reads the logits once more and computes what the one call does). A row whose weight is 0 takes no part: its logits are not read,
its loss and gradient are 0. Logits may have any leading dimensions and row stride; per-row
operands are float32, contiguous, one value per row. Work is enqueued on the current stream
of the logits' device.
"""

from __future__ import annotations

import torch

from . import binding as B
from .context import context, dtype_code, matrix, new_like, on_gpu, stream_of, vector, written


def _rows(logits, weights, temperature, out=None, loss=None, lse=None, lse_given=False, grad_rows=None):
    """(muon_logits, logits as rows x vocab, device) after the checks. ``lse``: the rows' pairs."""
    code = dtype_code(logits, "logits")
    device = on_gpu(logits, "logits")
    if logits.dim() < 1:
        raise ValueError("logits must have at least one dimension")
    z = logits if logits.dim() == 2 else logits.reshape(-1, logits.shape[-1])
    rows, vocab = z.shape
    f32 = torch.float32
    d = ld_d = None
    if out is not None:
        if out.shape != logits.shape:
            raise ValueError(f"out has shape {tuple(out.shape)}, the logits {tuple(logits.shape)}")
        o = out if out.dim() == 2 else out.view(-1, vocab)
        ld_d = matrix(o, "out", z.shape, logits.dtype, device)
        d = o.data_ptr()
    l = B.muon_logits(z.data_ptr(), d, None if weights is None else vector(weights, "weights", rows, f32, device),
                      None if grad_rows is None else vector(grad_rows, "grad_rows", rows, f32, device),
                      None if loss is None else loss.data_ptr(), None if lse is None else lse.data_ptr(),
                      matrix(z, "logits", z.shape, logits.dtype, device), ld_d or 0, rows, vocab, temperature, code,
                      int(lse_given), int(lse is not None))
    return l, z, device


def _policy(z, device, targets, old_logp, advantages, ref_logp, clip_low, clip_high, kl_coef, logp):
    rows, f32 = z.shape[0], torch.float32
    if kl_coef != 0.0 and ref_logp is None:
        raise ValueError("kl_coef needs ref_logp")
    return B.muon_policy(vector(targets, "targets", rows, torch.int64, device),
                         vector(old_logp, "old_logp", rows, f32, device),
                         vector(advantages, "advantages", rows, f32, device),
                         None if ref_logp is None else vector(ref_logp, "ref_logp", rows, f32, device),
                         None if logp is None else logp.data_ptr(), clip_low, clip_high, kl_coef)


def _distill(z, device, top_logits, top_ids, top_lse):
    rows = z.shape[0]
    t_code = dtype_code(top_logits, "top_logits")
    if not isinstance(top_ids, torch.Tensor) or top_ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("top_ids must be an int32 or int64 tensor")
    k = top_logits.shape[-1] if top_logits.dim() else 0
    if not 1 <= k <= B.MUON_MAX_TOP:
        raise ValueError(f"between 1 and {B.MUON_MAX_TOP} kept entries a row, got {k}")
    t2 = top_logits if top_logits.dim() == 2 else top_logits.reshape(-1, k)
    i2 = top_ids if top_ids.dim() == 2 else top_ids.reshape(-1, k)
    t = B.muon_distill(t2.data_ptr(), i2.data_ptr(),
                       None if top_lse is None else vector(top_lse, "top_lse", rows, torch.float32, device),
                       matrix(t2, "top_logits", (rows, k), t2.dtype, device),
                       matrix(i2, "top_ids", (rows, k), i2.dtype, device), k, t_code,
                       B.MUON_I64 if i2.dtype == torch.int64 else B.MUON_I32)
    return t, (t2, i2)


def _call(entry, name, device, l, t, top):
    ctx = context(device)
    nbytes = B.muon_loss_workspace_size(ctx, l, top)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    B.check(entry(ctx, l, t, ws.data_ptr() if nbytes else None, nbytes, stream_of(device)), name)


def policy_loss(logits, targets, old_logp, advantages, *, ref_logp=None, weights=None, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, temperature: float = 1.0, grad: bool = True, out=None):
    """(loss, logp, grad): the rows' weighted losses
    w (-min(rho A, clip(rho, 1 - clip_low, 1 + clip_high) A) + kl_coef (exp(d) - d - 1)),
    rho = exp(logp - old_logp), d = ref_logp - logp, the targets' log-probabilities, and the
    gradient of the losses' sum by the logits (None without ``grad``). A target outside the
    vocabulary takes no part, like weight 0."""
    lead = logits.shape[:-1]
    loss = torch.empty(lead, dtype=torch.float32, device=logits.device)
    logp = torch.empty(lead, dtype=torch.float32, device=logits.device)
    given = out if grad else None
    if grad and out is None:
        out = new_like(logits)
    l, z, device = _rows(logits, weights, temperature, out if grad else None, loss)
    t = _policy(z, device, targets, old_logp, advantages, ref_logp, clip_low, clip_high, kl_coef, logp)
    _call(B.muon_policy_loss, "muon_policy_loss", device, l, t, 0)
    written(given)
    return loss, logp, out if grad else None


def distill_loss(logits, top_logits, top_ids, *, top_lse=None, weights=None, temperature: float = 1.0,
                 grad: bool = True, out=None):
    """(loss, grad): the rows' weighted losses w sum_j p_j (log p_j - log q_{i_j}), with p the
    teacher's kept logits over the temperature, normalised by ``top_lse`` (the teacher's log
    sum exp of its logits / temperature over its whole vocabulary) or among themselves, and q
    the student's probabilities; and the gradient of the losses' sum by the logits (None
    without ``grad``). Entries with an id outside the vocabulary are absent."""
    loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=logits.device)
    given = out if grad else None
    if grad and out is None:
        out = new_like(logits)
    l, z, device = _rows(logits, weights, temperature, out if grad else None, loss)
    t, keep = _distill(z, device, top_logits, top_ids, top_lse)
    _call(B.muon_distill_loss, "muon_distill_loss", device, l, t, t.top)
    written(given)
    return loss, out if grad else None


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, old_logp, advantages, ref_logp, weights, clip_low, clip_high, kl_coef, temperature):
        new = lambda *n: torch.empty((*logits.shape[:-1], *n), dtype=torch.float32, device=logits.device)  # noqa: E731
        loss, logp, lse = new(), new(), new(2)
        l, z, device = _rows(logits, weights, temperature, None, loss, lse)
        t = _policy(z, device, targets, old_logp, advantages, ref_logp, clip_low, clip_high, kl_coef, logp)
        _call(B.muon_policy_loss, "muon_policy_loss", device, l, t, 0)
        ctx.save_for_backward(logits, targets, old_logp, advantages, ref_logp, weights, lse)
        ctx.numbers = (clip_low, clip_high, kl_coef, temperature)
        ctx.mark_non_differentiable(logp)
        return loss, logp

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss, _):
        logits, targets, old_logp, advantages, ref_logp, weights, lse = ctx.saved_tensors
        clip_low, clip_high, kl_coef, temperature = ctx.numbers
        out = new_like(logits)
        up = grad_loss.contiguous()
        l, z, device = _rows(logits, weights, temperature, out, None, lse, True, up)
        t = _policy(z, device, targets, old_logp, advantages, ref_logp, clip_low, clip_high, kl_coef, None)
        _call(B.muon_policy_loss, "muon_policy_loss", device, l, t, 0)
        return (out,) + (None,) * 9


def policy_loss_rows(logits, targets, old_logp, advantages, *, ref_logp=None, weights=None, clip_low: float = 0.2,
                     clip_high: float = 0.2, kl_coef: float = 0.0, temperature: float = 1.0):
    """(loss, logp) of ``policy_loss``; the losses are differentiable in the logits."""
    return _PolicyLoss.apply(logits, targets, old_logp, advantages, ref_logp, weights, clip_low, clip_high, kl_coef,
                             temperature)


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_logits, top_ids, top_lse, weights, temperature):
        new = lambda *n: torch.empty((*logits.shape[:-1], *n), dtype=torch.float32, device=logits.device)  # noqa: E731
        loss, lse = new(), new(2)
        l, z, device = _rows(logits, weights, temperature, None, loss, lse)
        t, keep = _distill(z, device, top_logits, top_ids, top_lse)
        _call(B.muon_distill_loss, "muon_distill_loss", device, l, t, t.top)
        ctx.save_for_backward(logits, top_logits, top_ids, top_lse, weights, lse)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss):
        logits, top_logits, top_ids, top_lse, weights, lse = ctx.saved_tensors
        out = new_like(logits)
        up = grad_loss.contiguous()
        l, z, device = _rows(logits, weights, ctx.temperature, out, None, lse, True, up)
        t, keep = _distill(z, device, top_logits, top_ids, top_lse)
        _call(B.muon_distill_loss, "muon_distill_loss", device, l, t, t.top)
        return (out,) + (None,) * 5


def distill_loss_rows(logits, top_logits, top_ids, *, top_lse=None, weights=None, temperature: float = 1.0):
    """The losses of ``distill_loss``, differentiable in the logits."""
    return _DistillLoss.apply(logits, top_logits, top_ids, top_lse, weights, temperature)
