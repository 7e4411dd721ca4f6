"""RMS norm with the residual's addition: the pre-norm of a block (argument marshalling only).

    s = x + residual,   y = weight * s / sqrt(mean(s^2) + eps)      over the last dimension

in fp32 whatever the types, s and y rounded once.  x is fp32, bf16 or fp16 [..., E] (rows may lie a
constant step apart, as in a slice of a wider tensor), the residual stream fp32 or x's type, the weight
fp32 [E].  ``forward_fp8`` returns y in e4m3 with scales, ``backward`` the gradient.  Every step runs in
the CUDA library; outputs belong to the call's stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native as nat
from ._call import TYPES, check_shape, check_tensor, on, ptr, raw_stream, token_stride, workspace as _ws

_IO = (torch.float32, torch.bfloat16, torch.float16)


def _forward(x, weight, residual, eps, fp8, block, y, residual_out, scales, stream):
    check_tensor("x", x, _IO, contiguous=False)
    if x.dim() < 1:
        raise ValueError("x must be [..., E]")
    dev, E = x.device, x.shape[-1]
    check_tensor("weight", weight, (torch.float32,), dev)
    check_shape("weight", weight, (E,))
    a = nat.FvRmsnormArgs()
    a.E, a.eps, a.block = E, float(eps), int(block)
    a.M = x.numel() // E if E else 0
    a.x_stride = token_stride("x", x, x.dim() - 1, 1)
    a.x_type = TYPES[x.dtype]
    a.y_type = nat.FV_TYPE_E4M3 if fp8 else a.x_type
    if residual is not None:
        check_tensor("residual", residual, {x.dtype, torch.float32}, dev)
        check_shape("residual", residual, x.shape)
        a.res_type = TYPES[residual.dtype]
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if fp8 and block not in (0, 128):
        raise ValueError("block must be 128, or 0 for one scale a row")
    if fp8 and block and E % block:
        raise ValueError(f"blocks of {block} channels need E a multiple of {block}, got {E}")
    with on(dev, stream):
        y_dtype = torch.float8_e4m3fn if fp8 else x.dtype
        if y is None:
            y = torch.empty(x.shape, dtype=y_dtype, device=dev)
        else:
            check_tensor("y", y, (y_dtype,), dev)
            check_shape("y", y, x.shape)
        if residual is not None:
            if residual_out is None:
                residual_out = torch.empty_like(residual)
            else:
                check_tensor("residual_out", residual_out, (residual.dtype,), dev)
                check_shape("residual_out", residual_out, x.shape)
        if fp8:
            shape = (*x.shape[:-1], E // block if block else 1)
            if scales is None:
                scales = torch.empty(shape, dtype=torch.float32, device=dev)
            else:
                check_tensor("scales", scales, (torch.float32,), dev)
                check_shape("scales", scales, shape)
        a.x, a.residual, a.weight, a.y, a.s, a.scales = (ptr(x), ptr(residual), ptr(weight), ptr(y), ptr(residual_out),
                                                         ptr(scales))
        nat.check(nat.lib().fastvim_rmsnorm_forward(ctypes.byref(a), raw_stream(dev)), "fastvim_rmsnorm_forward")
    return y, scales, residual_out


def forward(x, weight, residual=None, eps=1e-5, y=None, residual_out=None, stream=None):
    """Queue the norm on ``stream`` (default: the current stream) and return y, or (y, s) with a residual.
    ``residual_out`` may be the residual itself, which is then updated in place."""
    y, _, s = _forward(x, weight, residual, eps, False, 0, y, residual_out, None, stream)
    return y if residual is None else (y, s)


def forward_fp8(x, weight, residual=None, eps=1e-5, block=128, y=None, scales=None, residual_out=None, stream=None):
    """``forward`` with y in e4m3: returns (y, scales), or (y, scales, s) with a residual; y * scales stands
    for the norm.  block=128: scales [..., E / 128], one for each 128 channels; block=0: scales [..., 1], one
    a row."""
    y, scales, s = _forward(x, weight, residual, eps, True, block, y, residual_out, scales, stream)
    return (y, scales) if residual is None else (y, scales, s)


def backward_workspace_size(M, E) -> int:
    a = nat.FvRmsnormGradArgs()
    a.M, a.E = M, E
    n = int(nat.lib().fastvim_rmsnorm_backward_workspace_size(ctypes.byref(a)))
    if n == 0:
        nat.check(nat.FV_ERR_SHAPE, "fastvim_rmsnorm_backward_workspace_size")
    return n


def backward(s, weight, dy, ds=None, eps=1e-5, x_dtype=None, grads=None, workspace=None, stream=None) -> dict:
    """Queue the gradient and return {"dx", "dresidual", "dweight"}.  s is the forward's s (x without a
    residual), dy the gradient of y, ds the gradient that s receives from elsewhere in the network (added).
    x and the residual have one gradient: "dx" in x's type ``x_dtype`` (that of dy), "dresidual" in the type
    of s -- the same tensor where the types agree.  dweight sums over all rows in a fixed order."""
    check_tensor("s", s, _IO)
    dev, E = s.device, s.shape[-1] if s.dim() else 0
    check_tensor("dy", dy, _IO, dev)
    check_shape("dy", dy, s.shape)
    if x_dtype is not None and x_dtype != dy.dtype:
        raise TypeError(f"dy must have the type of x, {x_dtype}, got {dy.dtype}")
    if s.dtype not in (dy.dtype, torch.float32):
        raise TypeError(f"s must be {dy.dtype} or torch.float32, got {s.dtype}")
    check_tensor("weight", weight, (torch.float32,), dev)
    check_shape("weight", weight, (E,))
    if ds is not None:
        check_tensor("ds", ds, (s.dtype,), dev)
        check_shape("ds", ds, s.shape)
    a = nat.FvRmsnormGradArgs()
    a.M, a.E, a.eps = s.numel() // E if E else 0, E, float(eps)
    a.s_type, a.y_type = TYPES[s.dtype], TYPES[dy.dtype]
    with on(dev, stream):
        want = {"dx": (s.shape, dy.dtype), "dweight": (weight.shape, torch.float32)}
        if s.dtype != dy.dtype:
            want["dresidual"] = (s.shape, s.dtype)
        if grads is None:
            grads = {n: torch.empty(shape, dtype=t, device=dev) for n, (shape, t) in want.items()}
        for n, (shape, t) in want.items():
            check_tensor(n, grads.get(n), (t,), dev)
            check_shape(n, grads[n], shape)
        ws = _ws(workspace, backward_workspace_size(a.M, E) if workspace is None else 0, dev)
        a.s, a.dy, a.ds, a.weight = ptr(s), ptr(dy), ptr(ds), ptr(weight)
        a.dx, a.dresidual, a.dweight = ptr(grads["dx"]), ptr(grads.get("dresidual")), ptr(grads["dweight"])
        nat.check(nat.lib().fastvim_rmsnorm_backward(ctypes.byref(a), ptr(ws), ws.numel(), raw_stream(dev)),
                  "fastvim_rmsnorm_backward")
    return {"dx": grads["dx"], "dresidual": grads["dresidual" if s.dtype != dy.dtype else "dx"],
            "dweight": grads["dweight"]}
