"""RMS norm with the residual's addition: the pre-norm of a block (argument marshalling only).

    s = x + residual,   y = weight * s / sqrt(mean(s^2) + eps)      over the last dimension

in fp32 whatever the types, s and y rounded once.  x is fp32, bf16 or fp16 [..., E] (rows may lie a
constant step apart, as in a slice of a wider tensor), the residual stream fp32 or x's type, the weight
fp32 [E].  ``forward_fp8`` returns y in e4m3 with scales, ``backward`` the gradient.  Every step runs in
the CUDA library; outputs belong to the call's stream.
"""
from __future__ import annotations

from ctypes import byref

import torch

from . import _native as nat
from ._call import TYPES, check_tensor, count, need, need_tokens, on, out, ptr, raw_stream, workspace as _ws

_IO = (torch.float32, torch.bfloat16, torch.float16)
_F32, _F8 = torch.float32, torch.float8_e4m3fn


def _forward(x, weight, residual, eps, fp8, block, y, residual_out, scales, stream):
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype in TYPES):
        check_tensor("x", x, _IO, contiguous=False)
    shape, dtype, dev = x.shape, x.dtype, x.device
    if not shape:
        raise ValueError("x must be [..., E]")
    E = count("channels", shape[-1])
    a = nat.FvRmsnormArgs()
    a.weight = need("weight", weight, _F32, (E,), dev)
    if not x.is_contiguous():
        a.x_stride = need_tokens("x", x, dtype, shape, dev, len(shape) - 1, 1)
    a.M, a.E, a.eps, a.x = (x.numel() // E if E else 0), E, eps, x.data_ptr()
    a.x_type = a.y_type = TYPES[dtype]
    if residual is not None:
        if not isinstance(residual, torch.Tensor) or residual.dtype not in (dtype, _F32):
            check_tensor("residual", residual, (dtype, _F32), dev)
        a.residual = need("residual", residual, residual.dtype, shape, dev)
        a.res_type = TYPES[residual.dtype]
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if fp8:
        if block not in (0, 128):
            raise ValueError("block must be 128, or 0 for one scale a row")
        if block and E % block:
            raise ValueError(f"blocks of {block} channels need E a multiple of {block}, got {E}")
        a.y_type, a.block = nat.FV_TYPE_E4M3, block
    where = on(dev, stream)
    if where is None:
        return _queue(a, x, residual, fp8, y, residual_out, scales, dev)
    with where:
        return _queue(a, x, residual, fp8, y, residual_out, scales, dev)


def _queue(a, x, residual, fp8, y, residual_out, scales, dev):
    y = out("y", y, x, _F8 if fp8 else x.dtype, x.shape, dev)
    a.y = y.data_ptr()
    if residual is not None:
        residual_out = out("residual_out", residual_out, residual, residual.dtype, x.shape, dev)
        a.s = residual_out.data_ptr()
    if fp8:
        scales = out("scales", scales, None, _F32, (*x.shape[:-1], a.E // a.block if a.block else 1), dev)
        a.scales = scales.data_ptr()
    status = nat.lib().fastvim_rmsnorm_forward(byref(a), raw_stream(dev))
    if status:
        nat.check(status, "fastvim_rmsnorm_forward")
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
    a.M, a.E = M, count("channels", E)
    return _size(a)


def _size(a):
    n = int(nat.lib().fastvim_rmsnorm_backward_workspace_size(byref(a)))
    if n == 0:
        nat.check(nat.FV_ERR_SHAPE, "fastvim_rmsnorm_backward_workspace_size")
    return n


def backward(s, weight, dy, ds=None, eps=1e-5, x_dtype=None, grads=None, workspace=None, stream=None) -> dict:
    """Queue the gradient and return {"dx", "dresidual", "dweight"}.  s is the forward's s (x without a
    residual), dy the gradient of y, ds the gradient that s receives from elsewhere in the network (added).
    x and the residual have one gradient: "dx" in x's type ``x_dtype`` (that of dy), "dresidual" in the type
    of s -- the same tensor where the types agree and ``grads`` names no other.  dweight sums over all rows
    in a fixed order."""
    check_tensor("s", s, _IO)
    check_tensor("dy", dy, _IO)
    dev, shape = s.device, s.shape
    if not shape:
        raise ValueError("s must be [..., E]")
    E = count("channels", shape[-1])
    if x_dtype is not None and x_dtype != dy.dtype:
        raise TypeError(f"dy must have the type of x, {x_dtype}, got {dy.dtype}")
    if s.dtype not in (dy.dtype, _F32):
        raise TypeError(f"s must be {dy.dtype} or torch.float32, got {s.dtype}")
    a = nat.FvRmsnormGradArgs()
    a.s, a.dy, a.weight = s.data_ptr(), need("dy", dy, dy.dtype, shape, dev), need("weight", weight, _F32, (E,), dev)
    if ds is not None:
        a.ds = need("ds", ds, s.dtype, shape, dev)
    a.M, a.E, a.eps = (s.numel() // E if E else 0), E, eps
    a.s_type, a.y_type = TYPES[s.dtype], TYPES[dy.dtype]
    where = on(dev, stream)
    if where is None:
        return _queue_backward(a, s, weight, dy, grads or {}, workspace, dev)
    with where:
        return _queue_backward(a, s, weight, dy, grads or {}, workspace, dev)


def _queue_backward(a, s, weight, dy, grads, workspace, dev):
    dx = out("dx", grads.get("dx"), dy, dy.dtype, dy.shape, dev)
    dw = out("dweight", grads.get("dweight"), weight, _F32, weight.shape, dev)
    given = grads.get("dresidual")
    if s.dtype is dy.dtype and (given is None or given is dx):
        dr = None
    else:
        dr = out("dresidual", given, s, s.dtype, s.shape, dev)
    a.dx, a.dresidual, a.dweight = dx.data_ptr(), ptr(dr), dw.data_ptr()
    ws = _ws(workspace, _size(a) if workspace is None else 0, dev)
    nat.check(nat.lib().fastvim_rmsnorm_backward(byref(a), ws.data_ptr(), ws.numel(), raw_stream(dev)),
              "fastvim_rmsnorm_backward")
    return {"dx": dx, "dresidual": dx if dr is None else dr, "dweight": dw}
