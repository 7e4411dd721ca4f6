"""Linear attention with a decay for each head (argument marshalling only).

Per sequence and value head, with the key head of its group (Hk divides H):

    S_t = exp(g_t) S_{t-1} + k_t v_t^T        y_t = scale S_t^T q_t

``forward`` takes whole sequences, ``backward`` is its gradient, ``step`` advances kept states by one
token.  Dense: q, k [B,T,Hk,dk], v [B,T,H,dv]; packed: q, k [rows,Hk,dk], v [rows,H,dv] with cu_seqlens
int32 [N+1] on the device (sequence n is rows cu[n] .. cu[n+1]-1).  fp32 or bf16; g (log decays, fp32) is
[B,T,H] or [rows,H], or [H] for one decay a head.  States are fp32 [N,H,dk,dv].  q, k, v, g may be slices
of a wider tensor (tokens a constant step apart); outputs are contiguous and belong to the call's stream.
Every step runs in the CUDA library.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native as nat
from ._call import TYPES, check_shape, check_tensor, on, ptr, raw_stream, token_stride, workspace as _ws

_IO = (torch.float32, torch.bfloat16)


def _common(a, q, k, v, g, lead, scale):
    """Checks q, k, v, g (``lead`` token dimensions each) and fills sizes, strides and pointers of ``a``."""
    check_tensor("q", q, _IO, contiguous=False)
    dev = q.device
    for name, t in (("k", k), ("v", v)):
        check_tensor(name, t, (q.dtype,), dev, contiguous=False)
    check_tensor("g", g, (torch.float32,), dev, contiguous=False)
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dim() != lead + 2:
            raise ValueError(f"{name} must have {lead + 2} dimensions, got {list(t.shape)}")
    tokens = q.shape[:lead]
    Hk, dk = q.shape[lead:]
    H, dv = v.shape[lead:]
    check_shape("k", k, q.shape)
    check_shape("v", v, (*tokens, H, dv))
    if Hk == 0 or H % Hk:
        raise ValueError(f"the {Hk} key heads must divide the {H} value heads")
    if g.dim() == 1:
        check_shape("g", g, (H,))
        if not g.is_contiguous():
            raise ValueError("g must be contiguous")
        a.flags = nat.FV_LA_HEAD_DECAY
    else:
        check_shape("g", g, (*tokens, H))
        a.g_stride = token_stride("g", g, lead, 1)
    a.H, a.Hk, a.dk, a.dv, a.type = H, Hk, dk, dv, TYPES[q.dtype]
    a.scale = float(dk**-0.5 if scale is None else scale)
    a.q_stride, a.k_stride, a.v_stride = (token_stride(n, t, lead) for n, t in (("q", q), ("k", k), ("v", v)))
    a.q, a.k, a.v, a.g = ptr(q), ptr(k), ptr(v), ptr(g)
    return dev, tokens, H, dk, dv


def _sequences(a, q, k, v, g, scale, initial_state, cu_seqlens):
    lead = 2 if cu_seqlens is None else 1
    dev, tokens, H, dk, dv = _common(a, q, k, v, g, lead, scale)
    if cu_seqlens is None:
        a.N, a.T = tokens
    else:
        check_tensor("cu_seqlens", cu_seqlens, (torch.int32,), dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be [N+1]")
        a.N, a.T = cu_seqlens.numel() - 1, tokens[0]
        a.cu_seqlens = ptr(cu_seqlens)
    states = (a.N, H, dk, dv)
    if initial_state is not None:
        check_tensor("initial_state", initial_state, (torch.float32,), dev)
        check_shape("initial_state", initial_state, states)
        a.initial_state = ptr(initial_state)
    return dev, states


def _out(name, given, shape, dtype, dev):
    if given is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    check_tensor(name, given, (dtype,), dev)
    check_shape(name, given, shape)
    return given


def _size(fn, a):
    n = int(fn(ctypes.byref(a)))
    if n == 0:
        nat.check(nat.lib().fastvim_linattn_validate(ctypes.byref(a)), "fastvim_linattn_workspace_size")
    return n


def workspace_size(q, k, v, g, cu_seqlens=None) -> int:
    """Workspace bytes of ``forward`` on these tensors (by their sizes alone)."""
    a = nat.FvLinattnArgs()
    _sequences(a, q, k, v, g, None, None, cu_seqlens)
    return _size(nat.lib().fastvim_linattn_workspace_size, a)


def backward_workspace_size(q, k, v, g, cu_seqlens=None) -> int:
    """Workspace bytes of ``backward`` on these tensors (by their sizes alone)."""
    a = nat.FvLinattnArgs()
    _sequences(a, q, k, v, g, None, None, cu_seqlens)
    return _size(nat.lib().fastvim_linattn_backward_workspace_size, a)


def forward(q, k, v, g, scale=None, initial_state=None, cu_seqlens=None, return_state=False, y=None,
            final_state=None, workspace=None, stream=None):
    """Queue the attention on ``stream`` (default: the current stream) and return y, or (y, final_state) with
    return_state or a final_state buffer (which may be initial_state).  scale defaults to dk^-1/2.  Packed
    offsets that fall or leave the rows are found on the device: nothing is then written, and
    ``ssm.device_status`` of the workspace passed in tells."""
    a = nat.FvLinattnArgs()
    dev, states = _sequences(a, q, k, v, g, scale, initial_state, cu_seqlens)
    with on(dev, stream):
        y = _out("y", y, v.shape, v.dtype, dev)
        if return_state or final_state is not None:
            final_state = _out("final_state", final_state, states, torch.float32, dev)
        a.y, a.final_state = ptr(y), ptr(final_state)
        ws = _ws(workspace, _size(nat.lib().fastvim_linattn_workspace_size, a) if workspace is None else 0, dev)
        nat.check(nat.lib().fastvim_linattn_forward(ctypes.byref(a), ptr(ws), ws.numel(), raw_stream(dev)),
                  "fastvim_linattn_forward")
    return y if final_state is None else (y, final_state)


def backward(q, k, v, g, dy, scale=None, initial_state=None, d_final_state=None, cu_seqlens=None, grads=None,
             workspace=None, stream=None) -> dict:
    """Queue the gradient for the upstream gradients dy (of y) and d_final_state (of the final states; None:
    zero) and return {"dq", "dk", "dv", "dg"}, with "d_initial_state" where initial_state is given or the
    grads dict asks for it.  Everything is recomputed from the inputs; no forward workspace is needed.
    Gradients of shared key heads are summed over the value heads, a per-head g's over all tokens."""
    a = nat.FvLinattnArgs()
    dev, states = _sequences(a, q, k, v, g, scale, initial_state, cu_seqlens)
    check_tensor("dy", dy, (q.dtype,), dev, contiguous=False)
    check_shape("dy", dy, v.shape)
    a.dy_stride = token_stride("dy", dy, v.dim() - 2)
    if d_final_state is not None:
        check_tensor("d_final_state", d_final_state, (torch.float32,), dev)
        check_shape("d_final_state", d_final_state, states)
    with on(dev, stream):
        want = {"dq": (q.shape, q.dtype), "dk": (k.shape, q.dtype), "dv": (v.shape, q.dtype), "dg": (g.shape, torch.float32)}
        if initial_state is not None or (grads is not None and grads.get("d_initial_state") is not None):
            want["d_initial_state"] = (states, torch.float32)
        grads = {n: _out(n, None if grads is None else grads.get(n), shape, t, dev) for n, (shape, t) in want.items()}
        r = nat.FvLinattnGrads()
        r.dy, r.d_final_state = ptr(dy), ptr(d_final_state)
        for n, t in grads.items():
            setattr(r, n, ptr(t))
        ws = _ws(workspace, _size(nat.lib().fastvim_linattn_backward_workspace_size, a) if workspace is None else 0, dev)
        nat.check(nat.lib().fastvim_linattn_backward(ctypes.byref(a), ctypes.byref(r), ptr(ws), ws.numel(), raw_stream(dev)),
                  "fastvim_linattn_backward")
    return grads


def step(q, k, v, g, state, scale=None, slots=None, y=None, status=None, stream=None):
    """Queue one token of B sequences -- q, k [B,Hk,dk], v [B,H,dv], g [B,H] or [H] -- and return y [B,H,dv];
    ``state`` fp32 [S,H,dk,dv] is updated in place.  Row b uses state slots[b] (int32 [B]; a negative slot
    leaves the row out, its y is zero), or state b without slots.  A slot out of range, or one that an
    earlier row of the call has, is found on the device: the row's y is zero, no state changes for it, and
    ``status`` (an int32 tensor of one element, zeroed by the caller) receives FV_ERR_INDEX."""
    a = nat.FvLinattnStepArgs()
    dev, (B,), H, dk, dv = _common(a, q, k, v, g, 1, scale)
    check_tensor("state", state, (torch.float32,), dev)
    if state.dim() != 4:
        raise ValueError(f"state must be [S,H,dk,dv], got {list(state.shape)}")
    check_shape("state", state, (state.shape[0], H, dk, dv))
    a.B, a.S, a.state = B, state.shape[0], ptr(state)
    if slots is not None:
        check_tensor("slots", slots, (torch.int32,), dev)
        check_shape("slots", slots, (B,))
        a.slots = ptr(slots)
    elif a.S < B:
        raise ValueError(f"{B} rows need as many states, got {a.S}")
    if status is not None:
        check_tensor("status", status, (torch.int32,), dev)
        check_shape("status", status, (1,))
        a.status = ptr(status)
    with on(dev, stream):
        y = _out("y", y, v.shape, v.dtype, dev)
        a.y = ptr(y)
        nat.check(nat.lib().fastvim_linattn_step(ctypes.byref(a), raw_stream(dev)), "fastvim_linattn_step")
    return y
