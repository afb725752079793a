"""One library context per GPU for the operators that only read it (``layers``, ``losses``),
created on first use and kept for the process, and their argument checks."""

from __future__ import annotations

import threading

import torch

from . import binding as B

_contexts: dict = {}
_lock = threading.Lock()

DTYPE_CODES = {torch.float32: B.MUON_F32, torch.bfloat16: B.MUON_BF16}


def context(device: torch.device):
    ctx = _contexts.get(device.index)
    if ctx is None:
        with _lock:
            ctx = _contexts.get(device.index)
            if ctx is None:
                ctx = _contexts[device.index] = B.muon_init(device.index)
    return ctx


# The current stream's handle without a Stream object around it where torch has it (2 us less
# of the about 17 a small call takes on the host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def stream_of(device: torch.device) -> int:
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def new_like(t: torch.Tensor) -> torch.Tensor:
    """An uninitialised contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def written(*tensors) -> None:
    """Tells torch's automatic differentiation that a call has written given tensors (through
    their addresses, which it does not see): a node that saved one refuses its backward."""
    given = [t for t in tensors if t is not None]
    if given:
        torch.autograd.graph.increment_version(given)


def dtype_code(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    code = DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


def on_gpu(t: torch.Tensor, name: str) -> torch.device:
    if t.device.type != "cuda":
        raise ValueError(f"{name} is on {t.device}, not on a GPU")
    return t.device


def matrix(t: torch.Tensor, name: str, shape: tuple, dtype: torch.dtype, device: torch.device) -> int:
    """The row stride of a 2-D operand after its checks: type, device, shape, unit column
    stride, rows that do not overlap."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    rows, cols = shape
    if t.is_contiguous():
        return max(cols, 1)
    ld, step = t.stride()
    if rows and cols > 1 and step != 1:
        raise ValueError(f"{name} must have unit column stride, got strides {t.stride()}")
    if rows <= 1:
        return max(cols, 1)
    if ld < cols:
        raise ValueError(f"{name} has overlapping rows (strides {t.stride()}): make it contiguous")
    return ld


def vector(t: torch.Tensor, name: str, rows: int, dtype: torch.dtype, device: torch.device) -> int:
    """The address of a contiguous per-row operand after its checks."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.numel() != rows:
        raise ValueError(f"{name} has {t.numel()} elements, expected {rows}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()
