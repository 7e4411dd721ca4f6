"""What the bindings of the operators around the layer share: the device and stream of a call, and
the token strides of its tensors.  Argument marshalling only."""
from __future__ import annotations

import contextlib

import torch

from . import _native as nat

TYPES = {torch.float32: nat.FV_TYPE_F32, torch.bfloat16: nat.FV_TYPE_BF16, torch.float16: nat.FV_TYPE_F16}


def check_tensor(name, t, dtypes, device=None, contiguous=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def check_shape(name, t, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def token_stride(name, t, lead, inner=2) -> int:
    """Elements between tokens of ``t``, whose last ``inner`` dimensions are one token's values and must
    be dense, and whose first ``lead`` ones are the tokens, which must lie a constant step apart: a slice
    of a fused projection qualifies.  0 where ``t`` is contiguous."""
    if t.is_contiguous() or t.numel() == 0:
        return 0
    width = 1
    for d in range(t.dim() - 1, t.dim() - inner - 1, -1):
        if t.shape[d] != 1 and t.stride(d) != width:
            raise ValueError(f"{name}: the values of one token must be contiguous, got strides {t.stride()}")
        width *= t.shape[d]
    step = None
    for d in range(lead - 1, -1, -1):
        if t.shape[d] == 1:
            continue
        if step is None:
            step, rows = t.stride(d), t.shape[d]
        elif t.stride(d) != step * rows:
            raise ValueError(f"{name}: the tokens must lie a constant step apart, got strides {t.stride()}")
        else:
            rows *= t.shape[d]
    if step is None:
        return 0  # one token
    if step < width:
        raise ValueError(f"{name}: tokens overlap in memory (strides {t.stride()}); make it contiguous")
    return step


def on(device, stream):
    """A context in which allocations and launches belong to ``device`` and ``stream`` (default: the
    device's current stream): memory allocated inside is reused only after that stream's work."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)
    if torch.cuda.current_device() != device.index:
        return torch.cuda.device(device)
    return contextlib.nullcontext()


def raw_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


def workspace(given, size, device):
    """``given``, checked, or a new buffer of ``size`` bytes from the current stream's pool."""
    if given is None:
        return torch.empty(max(size, 256), dtype=torch.uint8, device=device)
    check_tensor("workspace", given, (torch.uint8,), device)
    return given


def ptr(t):
    return None if t is None else t.data_ptr()
