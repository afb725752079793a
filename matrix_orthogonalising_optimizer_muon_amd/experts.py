"""Tokens sorted by expert and back (``muon_expert_plan``, ``muon_expert_dispatch``,
``muon_expert_combine``, ``muon_expert_combine_backward``).

``expert_plan`` sorts the choices (token t's j-th expert, f = t top + j) by expert, stably.
``dispatch`` gathers the tokens' rows in that order, so that each expert's lie together;
``combine`` adds the experts' rows back to their tokens with weights. Both are differentiable;
``dispatch_forward`` / ``dispatch_backward`` and ``combine_forward`` / ``combine_backward`` are the
calls themselves. A choice outside [0, experts) is dropped: it has no row and adds nothing.
The sorted arrays always have tokens x top rows (nothing waits for the GPU); those behind the
last expert's are zeros. ``RoutedFeedForward`` runs a gated feed-forward block per expert between
the two. Work is enqueued on the current stream of the operands' device.
"""

from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import binding as B
from .context import context, dtype_code, matrix, on_gpu, stream_of, vector
from .layers import GatedFeedForward


@dataclass(frozen=True)
class ExpertPlan:
    """``order`` (tokens x top): the choice of each row, -1 behind the last; ``slots`` (as the ids):
    the row of each choice, -1 where it is dropped; ``offsets`` (experts + 1): each expert's
    first row, then their number. All int32 on the GPU."""
    order: torch.Tensor
    slots: torch.Tensor
    offsets: torch.Tensor
    tokens: int
    top: int
    experts: int

    def __post_init__(self):
        object.__setattr__(self, "_c", B.muon_experts(None, self.order.data_ptr(), self.slots.data_ptr(), self.offsets.data_ptr(),
                                                      self.tokens, self.top, self.experts, 0, 0))


def expert_plan(ids, experts: int) -> ExpertPlan:
    """The plan for ``ids``, each token's experts along the last axis (int32 or int64)."""
    if not isinstance(ids, torch.Tensor) or ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be an int32 or int64 tensor")
    device = on_gpu(ids, "ids")
    if ids.dim() < 1 or not 1 <= ids.shape[-1] <= B.MUON_MAX_CHOICES:
        raise ValueError(f"ids must have between 1 and {B.MUON_MAX_CHOICES} experts a token along the last axis, "
                         f"got shape {tuple(ids.shape)}")
    if not 1 <= experts <= B.MUON_MAX_EXPERTS:
        raise ValueError(f"between 1 and {B.MUON_MAX_EXPERTS} experts, got {experts}")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    top = ids.shape[-1]
    tokens = ids.numel() // top
    # one allocation for the three
    n = tokens * top
    both = torch.empty(2 * n + experts + 1, dtype=torch.int32, device=device)
    plan = ExpertPlan(both[:n], both[n:2 * n].view(ids.shape), both[2 * n:], tokens, top, experts)
    e = B.muon_experts.from_buffer_copy(plan._c)
    e.ids = ids.data_ptr()
    e.id_dtype = B.MUON_I64 if ids.dtype == torch.int64 else B.MUON_I32
    ctx = context(device)
    nbytes = B.muon_expert_plan_workspace_size(ctx, e)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    B.check(B.muon_expert_plan(ctx, e, ws.data_ptr() if nbytes else None, nbytes, stream_of(device)), "muon_expert_plan")
    return plan


def _rows(t, name, rows, plan, dim=None, dtype=None):
    """(t as rows x dim, its row stride, its type's code) after the checks."""
    code = dtype_code(t, name)
    if t.dim() < 1 or t.shape[-1] < 1 or (dim is not None and t.shape[-1] != dim):
        raise ValueError(f"{name} has shape {tuple(t.shape)}" + ("" if dim is None else f", expected {dim} columns"))
    t2 = t if t.dim() == 2 else t.reshape(-1, t.shape[-1])
    return t2, matrix(t2, name, (rows, t.shape[-1]), t.dtype if dtype is None else dtype, plan.slots.device), code


def _check_plan(plan):
    if not isinstance(plan, ExpertPlan):
        raise TypeError(f"plan must be what expert_plan returned, got {type(plan).__name__}")


def dispatch_forward(x, plan: ExpertPlan):
    """The tokens' rows in the plan's order: (tokens x top) x dim."""
    _check_plan(plan)
    x2, ld, code = _rows(x, "x", plan.tokens, plan)
    device, dim = x2.device, x2.shape[1]
    xs = torch.empty((plan.tokens * plan.top, dim), dtype=x2.dtype, device=device)
    B.check(B.muon_expert_dispatch(context(device), plan._c, x2.data_ptr(), ld, xs.data_ptr(), dim, dim,
                                   code, stream_of(device)), "muon_expert_dispatch")
    return xs


def _combine(rows, name, weights, plan):
    _check_plan(plan)
    r2, ld, code = _rows(rows, name, plan.tokens * plan.top, plan)
    device, dim = r2.device, r2.shape[1]
    w = None if weights is None else vector(weights, "weights", plan.tokens * plan.top, torch.float32, device)
    y = torch.empty((*plan.slots.shape[:-1], dim), dtype=r2.dtype, device=device)
    B.check(B.muon_expert_combine(context(device), plan._c, r2.data_ptr(), ld, w, y.data_ptr(), dim, dim,
                                  code, stream_of(device)), "muon_expert_combine")
    return y


def dispatch_backward(dxs, plan: ExpertPlan):
    """The gradient by x: each token's rows of ``dxs`` added up, in the shape of the ids with dim
    in the place of top."""
    return _combine(dxs, "dxs", None, plan)


def combine_forward(ys, weights, plan: ExpertPlan):
    """y[t] = sum_j weights[t, j] ys[slots[t, j]], in the shape of the ids with dim in the place of
    top. ``weights``: float32, as many as ids, or None: 1."""
    return _combine(ys, "ys", weights, plan)


def combine_backward(dy, ys, weights, plan: ExpertPlan, *, need=(True, True)):
    """(dys, dweights) for the gradient ``dy`` of y; ``need``: which of the two are wanted (None in
    the place of the other; ``ys`` may be None without the second)."""
    _check_plan(plan)
    dy2, ld, code = _rows(dy, "dy", plan.tokens, plan)
    device, dim, n = dy2.device, dy2.shape[1], plan.tokens * plan.top
    ys2, ld_ys, _ = _rows(ys, "ys", n, plan, dim, dy2.dtype) if need[1] else (None, dim, code)
    w = None if weights is None else vector(weights, "weights", n, torch.float32, device)
    dys = torch.empty((n, dim), dtype=dy2.dtype, device=device) if need[0] else None
    dw = torch.empty(plan.slots.shape, dtype=torch.float32, device=device) if need[1] else None
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    B.check(B.muon_expert_combine_backward(context(device), plan._c, dy2.data_ptr(), ld, ptr(ys2), ld_ys, w, ptr(dys),
                                           dim, ptr(dw), dim, code, stream_of(device)),
            "muon_expert_combine_backward")
    return dys, dw


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        ctx.save_for_backward(plan.order, plan.slots, plan.offsets)
        ctx.plan, ctx.shape = plan, x.shape
        return dispatch_forward(x, plan)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dxs):
        ctx.saved_tensors      # refused where the plan was written to
        return dispatch_backward(dxs.contiguous(), ctx.plan).view(ctx.shape), None


def dispatch(x, plan: ExpertPlan):
    """``dispatch_forward``, differentiable in x."""
    return _Dispatch.apply(x, plan)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, plan):
        # ys is read again for the weights' gradient alone
        want = weights is not None and ctx.needs_input_grad[1]
        ctx.save_for_backward(ys if want else None, weights, plan.order, plan.slots, plan.offsets)
        ctx.plan, ctx.shape = plan, ys.shape
        return combine_forward(ys, weights, plan)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        ys, weights, *_ = ctx.saved_tensors
        dys, dw = combine_backward(dy.contiguous(), ys, weights, ctx.plan, need=ctx.needs_input_grad[:2])
        return (None if dys is None else dys.view(ctx.shape)), (None if dw is None else dw.view(weights.shape)), None


def combine(ys, weights, plan: ExpertPlan):
    """``combine_forward``, differentiable in ys and weights."""
    return _Combine.apply(ys, weights, plan)


class RoutedFeedForward(torch.nn.Module):
    """A layer's feed-forward blocks behind a router: each token goes to the ``top`` experts of the
    largest scores x router^T, weighted by the softmax over those. ``router`` and the experts'
    ``gate``, ``up`` and ``down`` are matrices that ``MuonWithAdamW`` routes to the Muon update.
    A call waits for the number of each expert's tokens, which sizes the blocks' products, so it cannot be captured
    into a graph."""

    def __init__(self, dim: int, hidden: int, experts: int, top: int, *, activation: str = "silu", device=None,
                 dtype=torch.bfloat16):
        super().__init__()
        if not 1 <= top <= min(experts, B.MUON_MAX_CHOICES) or experts > B.MUON_MAX_EXPERTS:
            raise ValueError(f"top {top} of {experts} experts: at most {B.MUON_MAX_CHOICES} of {B.MUON_MAX_EXPERTS}, none twice")
        self.top = top
        self.router = torch.nn.Parameter(torch.randn(experts, dim, device=device, dtype=torch.float32)
                                         .mul_(1.0 / math.sqrt(dim)).to(dtype))
        self.experts = torch.nn.ModuleList(GatedFeedForward(dim, hidden, activation=activation, device=device, dtype=dtype)
                                           for _ in range(experts))

    def forward(self, x):
        chosen = (x.float() @ self.router.float().T).topk(self.top, dim=-1)
        plan = expert_plan(chosen.indices, len(self.experts))
        xs = dispatch(x, plan)
        first = plan.offsets.tolist()
        rows = xs.split([b - a for a, b in zip(first, first[1:])])
        ys = torch.cat([f(r) if r.shape[0] else r for f, r in zip(self.experts, rows)])
        return combine(ys, torch.softmax(chosen.values, dim=-1), plan)
