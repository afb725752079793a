"""Linear attention with a decay for each head (``muon_mix_forward``, ``muon_mix_backward``,
``muon_mix_step``): the mixer whose query, key, value and output matrices are the rest of a
decoder layer's Muon list. For batch entry b and head h, S a dim x dim_v state in float32:

    S <- exp(log_decay[h]) S + k_t^T v_t,   o_t = scale q_t S

q is batch x tokens x heads x dim, k batch x tokens x kv_heads x dim, v batch x tokens x kv_heads x
dim_v, all float32 or all bfloat16, with unit stride along the last axis and any others (views
of a joint projection or of heads-first arrays are read in place); query head h reads k, v head
h // (heads // kv_heads). The decay is a constant: it has no gradient.

``linear_attention_forward`` / ``linear_attention_backward`` are the two calls,
``linear_attention`` the same for torch's automatic differentiation, ``linear_attention_step``
one token of every sequence. ``state`` (batch x heads x dim x dim_v, float32, contiguous) carries a
sequence on; ``lengths`` (int32, on the GPU) gives each sequence of a padded batch its tokens:
what lies behind is not read, its outputs and gradients are zeros. Work is enqueued on the
current stream of the operands' device; workspaces come from torch's allocator for the
length of the call.
"""

from __future__ import annotations

import math

import torch

from . import binding as B
from .context import context, dtype_code, on_gpu, stream_of, vector, written


def _strides(t, name, lead, dtype, device, last):
    """The strides of an operand but for its last axis, after its checks."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != (*lead, last):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(*lead, last)}")
    *s, step = t.stride()
    if last > 1 and step != 1 and t.numel():
        raise ValueError(f"{name} must have unit stride along its last axis, got strides {t.stride()}")
    return tuple(s)


def _state(t, name, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != torch.float32:
        raise TypeError(f"{name} has dtype {t.dtype}, expected torch.float32")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _check_sizes(heads, kv_heads, dim, dim_v):
    if kv_heads < 1 or heads % kv_heads:
        raise ValueError(f"{heads} heads of q for {kv_heads} of k and v: not a multiple")
    if not (1 <= dim <= B.MUON_MIX_MAX_DIM and 1 <= dim_v <= B.MUON_MIX_MAX_DIM):
        raise ValueError(f"dim and dim_v must be between 1 and {B.MUON_MIX_MAX_DIM}, got {dim} and {dim_v}")


def _problem(q, k, v, log_decay, scale, state, lengths):
    """(muon_mix, device, shape of the states, shape of o) after the checks."""
    code = dtype_code(q, "q")
    device = on_gpu(q, "q")
    if q.dim() != 4 or not isinstance(k, torch.Tensor) or k.dim() != 4 or not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("q, k and v must be batch x tokens x heads x dim")
    batch, tokens, heads, dim = q.shape
    kv_heads, dim_v = v.shape[2:]
    _check_sizes(heads, kv_heads, dim, dim_v)
    if scale is None:
        scale = 1.0 / math.sqrt(dim)
    shape = (batch, heads, dim, dim_v)
    m = B.muon_mix(q.data_ptr(), k.data_ptr(), v.data_ptr(), vector(log_decay, "log_decay", heads, torch.float32, device),
                   None if state is None else _state(state, "state", shape, device),
                   None if lengths is None else vector(lengths, "lengths", batch, torch.int32, device),
                   _strides(q, "q", (batch, tokens, heads), q.dtype, device, dim),
                   _strides(k, "k", (batch, tokens, kv_heads), q.dtype, device, dim),
                   _strides(v, "v", (batch, tokens, kv_heads), q.dtype, device, dim_v),
                   batch, tokens, heads, kv_heads, dim, dim_v, scale, code)
    return m, device, shape, (batch, tokens, heads, dim_v)


def linear_attention_forward(q, k, v, log_decay, *, scale: float | None = None, state=None, lengths=None,
                             final: bool = False):
    """(o, states): o is batch x tokens x heads x dim_v; states (with ``final``, else None) those after
    each sequence's last token. ``scale``: 1 / sqrt(dim) where none is given."""
    m, device, shape, o_shape = _problem(q, k, v, log_decay, scale, state, lengths)
    o = torch.empty(o_shape, dtype=q.dtype, device=device)
    last = torch.empty(shape, dtype=torch.float32, device=device) if final else None
    ctx = context(device)
    nbytes = B.muon_mix_workspace_size(ctx, m)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    B.check(B.muon_mix_forward(ctx, m, o.data_ptr(), last.data_ptr() if final else None, ws.data_ptr() if nbytes else None,
                               nbytes, stream_of(device)), "muon_mix_forward")
    return o, last


def linear_attention_backward(do, q, k, v, log_decay, *, scale: float | None = None, state=None, lengths=None,
                              d_final=None, need_dstate: bool = False, need=(True, True, True)):
    """(dq, dk, dv, dstate) for the gradients ``do`` of o and ``d_final`` (None: zeros) of the last
    states. ``need``: which of dq, dk, dv are wanted (None in the place of the others); dstate with
    ``need_dstate``. Nothing of the forward is needed but its operands."""
    m, device, shape, o_shape = _problem(q, k, v, log_decay, scale, state, lengths)
    strides = _strides(do, "do", o_shape[:3], q.dtype, device, o_shape[3])
    outs = [torch.empty(t.shape, dtype=t.dtype, device=device) if n else None for t, n in zip((q, k, v), need)]
    ds = torch.empty(shape, dtype=torch.float32, device=device) if need_dstate else None
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    g = B.muon_mix_grads(do.data_ptr(), strides, None if d_final is None else _state(d_final, "d_final", shape, device),
                         *(ptr(t) for t in outs), ptr(ds))
    ctx = context(device)
    nbytes = B.muon_mix_workspace_size(ctx, m, g)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    B.check(B.muon_mix_backward(ctx, m, g, ptr(ws), nbytes, stream_of(device)), "muon_mix_backward")
    return (*outs, ds)


def linear_attention_step(q, k, v, log_decay, state, *, scale: float | None = None, out_state=None):
    """(o, states) of one token: q is batch x heads x dim, k batch x kv_heads x dim, v batch x kv_heads x
    dim_v, o batch x heads x dim_v. The new states go to ``out_state``, or replace ``state``."""
    code = dtype_code(q, "q")
    device = on_gpu(q, "q")
    if q.dim() != 3 or not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("q, k and v must be batch x heads x dim")
    batch, heads, dim = q.shape
    kv_heads, dim_v = v.shape[1:]
    _check_sizes(heads, kv_heads, dim, dim_v)
    if state is None:
        raise ValueError("a step needs the states")
    shape = (batch, heads, dim, dim_v)
    # (batch, head) strides; the token's is not read
    (qb, qh), (kb, kh), (vb, vh) = (_strides(q, "q", (batch, heads), q.dtype, device, dim),
                                    _strides(k, "k", (batch, kv_heads), q.dtype, device, dim),
                                    _strides(v, "v", (batch, kv_heads), q.dtype, device, dim_v))
    m = B.muon_mix(q.data_ptr(), k.data_ptr(), v.data_ptr(), vector(log_decay, "log_decay", heads, torch.float32, device),
                   _state(state, "state", shape, device), None, (qb, 0, qh), (kb, 0, kh), (vb, 0, vh), batch, 1, heads,
                   kv_heads, dim, dim_v, 1.0 / math.sqrt(dim) if scale is None else scale, code)
    new = state if out_state is None else out_state
    to = m.state if out_state is None else _state(new, "out_state", shape, device)
    o = torch.empty((batch, heads, dim_v), dtype=q.dtype, device=device)
    B.check(B.muon_mix_step(context(device), m, o.data_ptr(), to, stream_of(device)), "muon_mix_step")
    written(new)
    return o, new


class _LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, state, lengths, scale, final):
        o, last = linear_attention_forward(q, k, v, log_decay, scale=scale, state=state, lengths=lengths, final=final)
        ctx.save_for_backward(q, k, v, log_decay, state, lengths)
        ctx.scale = scale
        return (o, last) if final else o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do, d_final=None):
        q, k, v, log_decay, state, lengths = ctx.saved_tensors
        need = ctx.needs_input_grad
        # an expanded gradient (of a sum) has no unit stride of its own
        do = do if do.stride(-1) == 1 or do.shape[-1] == 1 else do.contiguous()
        out = linear_attention_backward(do, q, k, v, log_decay, scale=ctx.scale, state=state, lengths=lengths,
                                        d_final=None if d_final is None else d_final.contiguous(), need=need[:3],
                                        need_dstate=need[4])
        return (*out[:3], None, out[3], None, None, None)


def linear_attention(q, k, v, log_decay, *, scale: float | None = None, state=None, lengths=None, final: bool = False):
    """o, or with ``final`` (o, states), differentiable in q, k, v and ``state``."""
    if isinstance(log_decay, torch.Tensor) and log_decay.requires_grad and torch.is_grad_enabled():
        raise ValueError("log_decay is a constant here: it may not require a gradient")
    return _LinearAttention.apply(q, k, v, log_decay, state, lengths, scale, final)


class DecayAttention(torch.nn.Module):
    """A layer's mixer: the ``query``, ``key``, ``value`` and ``out`` matrices, which ``MuonWithAdamW``
    routes to the Muon update, around ``linear_attention``. Head h of n forgets with
    exp(log_decay[h]) = 1 - 2^-(5 + 7 h / (n - 1)) unless ``log_decay`` is given. ``log_decay`` stays
    float32 when the module is cast."""

    def __init__(self, dim: int, heads: int, head_dim: int, *, kv_heads: int | None = None, head_dim_v: int | None = None,
                 log_decay=None, device=None, dtype=torch.bfloat16):
        super().__init__()
        self.heads, self.kv_heads = heads, heads if kv_heads is None else kv_heads
        self.head_dim, self.head_dim_v = head_dim, head_dim if head_dim_v is None else head_dim_v
        if self.kv_heads < 1 or heads % self.kv_heads:
            raise ValueError(f"{heads} heads for {self.kv_heads} of k and v: not a multiple")

        def weight(rows, cols):
            return torch.nn.Parameter(torch.randn(rows, cols, device=device, dtype=torch.float32)
                                      .mul_(1.0 / math.sqrt(cols)).to(dtype))

        self.query, self.key = weight(heads * head_dim, dim), weight(self.kv_heads * head_dim, dim)
        self.value, self.out = weight(self.kv_heads * self.head_dim_v, dim), weight(dim, heads * self.head_dim_v)
        if log_decay is None:
            log_decay = torch.log1p(-torch.exp2(-5.0 - 7.0 * torch.arange(heads, dtype=torch.float32) / max(heads - 1, 1)))
        self.register_buffer("log_decay", torch.as_tensor(log_decay, dtype=torch.float32).detach().to(device).clone())

    def _apply(self, fn, recurse=True):
        kept = self.log_decay
        super()._apply(fn, recurse)
        # moved as the module is, but not cast: 8 bits would leave 1 - 2^-12 at 1
        self.log_decay = self.log_decay.float() if kept.is_meta else kept.to(self.log_decay.device)
        return self

    def _project(self, x):
        heads = lambda w, d: torch.nn.functional.linear(x, w).unflatten(-1, (-1, d))  # noqa: E731
        return heads(self.query, self.head_dim), heads(self.key, self.head_dim), heads(self.value, self.head_dim_v)

    def forward(self, x, *, state=None, lengths=None, final: bool = False):
        """y for x (batch x tokens x dim), or with ``final`` (y, states)."""
        got = linear_attention(*self._project(x), self.log_decay, state=state, lengths=lengths, final=final)
        o, last = got if final else (got, None)
        y = torch.nn.functional.linear(o.flatten(-2), self.out)
        return (y, last) if final else y

    @torch.no_grad()
    def step(self, x, state):
        """y for one token of every sequence, x batch x dim; ``state`` moves on in place."""
        o, _ = linear_attention_step(*self._project(x), self.log_decay, state)
        return torch.nn.functional.linear(o.flatten(-2), self.out)
