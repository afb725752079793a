"""The gated feed-forward block (``muon_ffn_forward`` / ``muon_ffn_backward``): the three
hidden matrices of a decoder layer that the Muon update spends most of its elements on.

    y = (act(x w_gate^T) * (x w_up^T)) w_down^T

``ffn_forward`` / ``ffn_backward`` are the two calls; the backward can write or accumulate
the weight gradients into given buffers, such as the persistent G arrays of a
``MuonUpdate``. ``gated_ffn`` is the same block for torch's automatic differentiation and
``GatedFeedForward`` a module holding the weights as ``gate``, ``up`` and ``down``, which
``MuonWithAdamW`` routes to the Muon update. Work is enqueued on the current stream of the
operands' device; workspaces come from torch's allocator for the length of the call. All of
them can be captured into a graph after one eager call; a backward through ``gated_ffn`` is
captured with ``torch.autograd.grad`` or with no eager graph of the same leaves alive, as
torch's own functions need it.
"""

from __future__ import annotations

import math

import torch

from . import binding as B
from .context import context, dtype_code, matrix, new_like, on_gpu, stream_of, written


def _block(x, w_gate, w_up, w_down, activation):
    """(muon_ffn, x as tokens x dim, device) after the checks."""
    code = dtype_code(x, "x")
    device = on_gpu(x, "x")
    if x.dim() < 1 or not isinstance(w_gate, torch.Tensor) or w_gate.dim() != 2:
        raise ValueError("x must have at least one dimension and w_gate two")
    if activation not in B.ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(B.ACTIVATIONS)}, got {activation!r}")
    hidden, dim = w_gate.shape
    if x.shape[-1] != dim:
        raise ValueError(f"x has {x.shape[-1]} columns, w_gate {dim}")
    x2 = x if x.dim() == 2 else x.reshape(-1, dim)
    dt = x.dtype
    f = B.muon_ffn(x2.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
                   matrix(x2, "x", x2.shape, dt, device), matrix(w_gate, "w_gate", w_gate.shape, dt, device),
                   matrix(w_up, "w_up", w_gate.shape, dt, device), matrix(w_down, "w_down", (dim, hidden), dt, device),
                   x2.shape[0], dim, hidden, code, B.ACTIVATIONS[activation])
    return f, x2, device


def ffn_forward(x, w_gate, w_up, w_down, *, activation: str = "silu", save: bool = False):
    """(y, saved): y has x's shape; ``saved`` (with ``save``) is what ``ffn_backward`` needs of
    the forward, a float32 tensor of g and u, else None."""
    f, x2, device = _block(x, w_gate, w_up, w_down, activation)
    y = new_like(x)
    ctx = context(device)
    nbytes, nsaved = B.muon_ffn_workspace_size(ctx, f)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    saved = torch.empty(nsaved // 4, dtype=torch.float32, device=device) if save else None
    B.check(B.muon_ffn_forward(ctx, f, y.data_ptr(), f.dim, saved.data_ptr() if save else None, ws.data_ptr(), nbytes,
                               stream_of(device)), "muon_ffn_forward")
    return y, saved


def _spans(tensors):
    """(first byte, last byte + 1, row stride, row width) of 2-D tensors with elements."""
    out = []
    for t in tensors:
        if t is not None and t.numel():
            es, (rows, cols), p = t.element_size(), t.shape, t.data_ptr()
            ld = t.stride(0) if rows > 1 else cols
            out.append((p, p + ((rows - 1) * ld + cols) * es, ld * es, cols * es))
    return out


def _overlap(a, b):
    if a[1] <= b[0] or b[1] <= a[0]:
        return False
    if a[2] != b[2]:
        return True
    # rows of one stride: apart when the columns lie side by side
    shift = (b[0] - a[0]) % a[2]
    return shift < a[3] or shift + b[3] > a[2]


def ffn_backward(dy, x, w_gate, w_up, w_down, saved, *, activation: str = "silu", grads=None,
                 accumulate: bool = False, need_dx: bool = True):
    """(dx, g_gate, g_up, g_down) for the gradient ``dy`` of y. ``grads``: (g_gate, g_up,
    g_down) buffers of the weights' shapes, all float32 or all bfloat16, that receive the
    weight gradients (with ``accumulate`` they are added to what is there); an entry may be
    None when that gradient is not wanted. They may not share memory with each other or with
    an operand. Without ``grads`` all three are new tensors of the weights' dtype."""
    return _backward(dy, x, w_gate, w_up, w_down, saved, activation, grads, accumulate, need_dx, grads is not None)


def _backward(dy, x, w_gate, w_up, w_down, saved, activation, grads, accumulate, need_dx, given_buffers):
    f, x2, device = _block(x, w_gate, w_up, w_down, activation)
    dy2 = dy if dy.dim() == 2 else dy.reshape(-1, f.dim)
    shapes = (w_gate.shape, w_up.shape, w_down.shape)
    if grads is None:
        if accumulate:
            raise ValueError("accumulate needs the gradient buffers (grads)")
        grads = (new_like(w_gate), new_like(w_up), new_like(w_down))
    names = ("g_gate", "g_up", "g_down")
    given = [t for t in grads if t is not None]
    g_code = dtype_code(given[0], "grads") if given else B.MUON_F32
    lds = [0 if t is None else matrix(t, n, s, given[0].dtype, device) for t, n, s in zip(grads, names, shapes)]
    if not isinstance(saved, torch.Tensor) or saved.dtype != torch.float32 or saved.device != device:
        raise TypeError("saved must be the float32 tensor ffn_forward(save=True) returned")
    if not saved.is_contiguous():
        raise ValueError("saved must be contiguous")
    ld_dy = matrix(dy2, "dy", x2.shape, x.dtype, device)
    if given_buffers:
        outs, ins = _spans(grads), _spans((dy2, x2, w_gate, w_up, w_down, saved.view(1, -1)))
        if any(_overlap(o, t) for i, o in enumerate(outs) for t in ins + outs[:i]):
            raise ValueError("the gradient buffers (grads) overlap each other or an operand")
    dx = new_like(x) if need_dx else None
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    g = B.muon_ffn_grads(dy2.data_ptr(), saved.data_ptr(), ptr(dx), *(ptr(t) for t in grads),
                         ld_dy, f.dim, *lds, g_code, int(accumulate))
    ctx = context(device)
    nbytes, nsaved = B.muon_ffn_workspace_size(ctx, f, g)
    if saved.numel() * 4 != nsaved:
        raise ValueError(f"saved has {saved.numel()} elements, this block's forward wrote {nsaved // 4}")
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    B.check(B.muon_ffn_backward(ctx, f, g, ws.data_ptr(), nbytes, stream_of(device)), "muon_ffn_backward")
    if given_buffers:
        written(*grads)
    return (dx, *grads)


class _GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, activation, grad_mode):
        # needs_input_grad names what requires a gradient also where no backward can come
        save = grad_mode and any(ctx.needs_input_grad)
        y, saved = ffn_forward(x, w_gate, w_up, w_down, activation=activation, save=save)
        ctx.save_for_backward(x, w_gate, w_up, w_down, saved)
        ctx.activation = activation
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w_gate, w_up, w_down, saved = ctx.saved_tensors
        need = ctx.needs_input_grad
        weights = (w_gate, w_up, w_down)
        grads = tuple(new_like(w) if n else None
                      for w, n in zip(weights, need[1:4]))
        # an expanded dy (of a sum) has no row stride of its own
        out = _backward(dy.contiguous(), x, *weights, saved, ctx.activation, grads, False, need[0], False)
        return (*out, None, None)


def gated_ffn(x, w_gate, w_up, w_down, activation: str = "silu"):
    """y of the block, differentiable in x and the three weights."""
    return _GatedFFN.apply(x, w_gate, w_up, w_down, activation, torch.is_grad_enabled())


class GatedFeedForward(torch.nn.Module):
    def __init__(self, dim: int, hidden: int, *, activation: str = "silu", device=None, dtype=torch.bfloat16):
        super().__init__()
        if activation not in B.ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(B.ACTIVATIONS)}, got {activation!r}")
        self.activation = activation

        def weight(rows, cols):
            return torch.nn.Parameter(torch.randn(rows, cols, device=device, dtype=torch.float32)
                                      .mul_(1.0 / math.sqrt(cols)).to(dtype))

        self.gate, self.up, self.down = weight(hidden, dim), weight(hidden, dim), weight(dim, hidden)

    def forward(self, x):
        return gated_ffn(x, self.gate, self.up, self.down, self.activation)
