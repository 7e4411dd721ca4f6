"""What the bindings of the operators around the layer share: checks of their tensors, the device and
stream of a call, and the token strides of its inputs.  Argument marshalling only.

The checks run on every call, so each has a short path for what a program passes normally (a plain
contiguous tensor of the right type and shape), and a long one that names what is wrong.
"""
from __future__ import annotations

import torch
from torch import Tensor

from . import _native as nat

TYPES = {torch.float32: nat.FV_TYPE_F32, torch.bfloat16: nat.FV_TYPE_BF16, torch.float16: nat.FV_TYPE_F16}


def check_tensor(name, t, dtypes, device=None, contiguous=True):
    if not isinstance(t, Tensor):
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


def count(name, n):
    """A size that the library takes in 32 bits."""
    if n >= 1 << 31:
        raise ValueError(f"{name} must be below 2^31, got {n}")
    return n


def need(name, t, dtype, shape, device):
    """``t`` is a contiguous tensor of this type and shape on ``device``; returns its address."""
    if not (type(t) is Tensor and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device):
        check_tensor(name, t, (dtype,), device)
        check_shape(name, t, shape)
    return t.data_ptr()


def need_tokens(name, t, dtype, shape, device, lead, inner=2):
    """As ``need``, with tokens (``lead`` dimensions) that may lie a constant step apart; returns the step."""
    if type(t) is Tensor and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return 0
    check_tensor(name, t, (dtype,), device, contiguous=False)
    check_shape(name, t, shape)
    return token_stride(name, t, lead, inner)


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
    """None where the call belongs to the current stream of the current device; else a context in which its
    allocations and launches belong to ``device`` and ``stream``: memory allocated inside is reused only
    after that stream's work."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream)
    if torch.cuda.current_device() != device.index:
        return torch.cuda.device(device)
    return None


# The raw handle of a device's current stream: PyTorch's own accessor where it has one (the public way
# builds a Stream object, 2 us of a call).
_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def raw_stream(device):
    return _raw(device.index) if _raw is not None else torch.cuda.current_stream(device).cuda_stream


def out(name, given, like, dtype, shape, device):
    """``given``, checked, or a new contiguous tensor; ``like``: one of the same shape, or None."""
    if given is not None:
        need(name, given, dtype, shape, device)
        return given
    if like is not None and like.is_contiguous():
        return torch.empty_like(like) if like.dtype is dtype else torch.empty_like(like, dtype=dtype)
    return torch.empty(shape, dtype=dtype, device=device)


def workspace(given, size, device):
    """``given``, checked, or a new buffer of ``size`` bytes from the current stream's pool."""
    if given is None:
        return torch.empty(max(size, 256), dtype=torch.uint8, device=device)
    check_tensor("workspace", given, (torch.uint8,), device)
    return given


def ptr(t):
    return None if t is None else t.data_ptr()
