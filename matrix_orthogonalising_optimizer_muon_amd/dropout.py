"""Dropout from a counter-based generator (``muon_dropout``): the mask is a function of a seed, an
offset and an element's number, so nothing of it is stored and the gradient draws it again.

    out = residual + keep x / (1 - p)        (p rounded to 1 / 65536)

``seed`` is an integer and ``offset`` another (a call's number, so that each call has a mask of its
own), or ``seed`` is a tensor of the two on the GPU (int64), read when the work runs: a captured
graph's replays then differ as the tensor does. ``dropout_forward`` / ``dropout_backward`` are the
calls, ``dropout`` the same for torch's automatic differentiation, ``Dropout`` a module that takes
its numbers from torch's generator or counts its calls. x may have any leading dimensions and row stride. Work is enqueued on the current
stream of the operands' device.
"""

from __future__ import annotations

import torch

from . import binding as B
from .context import context, dtype_code, matrix, new_like, on_gpu, stream_of, vector, written

_WORD = (1 << 64) - 1


def _number(v, name):
    if not isinstance(v, int):
        raise TypeError(f"{name} must be an integer, got {type(v).__name__}")
    if not -(1 << 63) <= v <= _WORD:
        raise ValueError(f"{name} must fit 64 bits, got {v}")
    return v & _WORD


def _call(x, p, seed, offset, residual, out):
    code = dtype_code(x, "x")
    device = on_gpu(x, "x")
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be between 0 and 1, got {p}")
    counter = None
    if isinstance(seed, torch.Tensor):
        counter = vector(seed, "seed", 2, torch.int64, device)
        if offset != 0:
            raise ValueError("the offset is the second entry of a seed tensor")
        seed = 0
    if residual is not None and isinstance(residual, torch.Tensor) and residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, x {tuple(x.shape)}")
    if out is not None and isinstance(out, torch.Tensor) and out.shape != x.shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, x {tuple(x.shape)}")
    given = out
    if out is None:
        out = new_like(x)
    cols = x.shape[-1] if x.dim() else 1

    def rows(t, name, view=False):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
        t2 = t if t.dim() == 2 else t.view(-1, cols) if view else t.reshape(-1, cols)
        return t2, matrix(t2, name, x2.shape, x.dtype, device)

    seed, offset = _number(seed, "seed"), _number(offset, "offset")
    if x.numel() == 0:
        return out
    x2 = x if x.dim() == 2 else x.reshape(-1, cols)
    _, ld_x = rows(x2, "x")
    r2, ld_r = rows(residual, "residual") if residual is not None else (None, 0)
    o2, ld_o = rows(out, "out", True)
    d = B.muon_drop(x2.data_ptr(), None if r2 is None else r2.data_ptr(), o2.data_ptr(), counter, ld_x, ld_r, ld_o, *x2.shape,
                    seed, offset, p, code)
    B.check(B.muon_dropout(context(device), d, stream_of(device)), "muon_dropout")
    written(given)
    return out


def dropout_forward(x, p: float, seed, offset: int = 0, *, residual=None, out=None):
    """residual + keep x / (1 - p), to ``out`` (which may be x or the residual) or a new tensor."""
    return _call(x, p, seed, offset, residual, out)


def dropout_backward(dy, p: float, seed, offset: int = 0, *, out=None):
    """The gradient by x for the gradient ``dy`` of the same call's output (the residual's is ``dy``)."""
    return _call(dy, p, seed, offset, None, out)


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset):
        ctx.p, ctx.offset = p, offset
        ctx.seed = None if isinstance(seed, torch.Tensor) else seed
        if ctx.seed is None:
            ctx.save_for_backward(seed)
        return dropout_forward(x, p, seed, offset, residual=residual)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        seed = ctx.saved_tensors[0] if ctx.seed is None else ctx.seed
        dx = dropout_backward(dy.contiguous(), ctx.p, seed, ctx.offset) if ctx.needs_input_grad[0] else None
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None


def dropout(x, p: float, seed, offset: int = 0, *, residual=None):
    """``dropout_forward``, differentiable in x and the residual. A seed tensor must keep its values
    until the backward."""
    return _Dropout.apply(x, residual, p, seed, offset)


class Dropout(torch.nn.Module):
    """``dropout`` with numbers of its own for each call; in evaluation x passes through (plus the residual).

    Without a seed every call draws both numbers from torch's generator of x's device: modules, their copies and
    differently seeded ranks have masks of their own, ``torch.manual_seed`` repeats them, replays of a captured
    graph differ, and activation checkpointing, which sets the generator back, draws a call's mask again.

    With a seed the numbers are it and a count of the module's calls, held on the GPU (``counter``): also the replays
    of a captured graph go on counting. Modules of one seed (copies too, and ranks, whose buffers
    DistributedDataParallel makes alike) draw the same masks. A call inside a backward is refused: a forward that
    activation checkpointing runs again there would have the next count's mask; ``dropout`` with the call's
    own offset runs again as it was."""

    def __init__(self, p: float, seed: int | None = None, *, device=None):
        super().__init__()
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"p must be between 0 and 1, got {p}")
        self.p = p
        if seed is not None:
            seed = _number(seed, "seed")
            seed = torch.tensor([seed - (1 << 64) if seed >> 63 else seed, 0], dtype=torch.int64, device=device)
        self.register_buffer("counter", seed)

    def forward(self, x, residual=None):
        if not self.training or self.p == 0.0:
            return x if residual is None else x + residual
        if self.counter is None:
            return dropout(x, self.p, torch.empty(2, dtype=torch.int64, device=x.device).random_(), residual=residual)
        if torch._C._current_graph_task_id() != -1:      # a backward is running on this thread
            raise RuntimeError("Dropout with a seed counts its calls, so its forward cannot be run again in a backward "
                               "(activation checkpointing): give it no seed, or call dropout(x, p, seed, offset) there")
        now = self.counter.clone()
        self.counter[1:].add_(1)
        return dropout(x, self.p, now, residual=residual)
