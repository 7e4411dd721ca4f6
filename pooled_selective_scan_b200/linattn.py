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

from ctypes import byref

import torch
from torch import Tensor

from . import _native as nat
from ._call import check_tensor, count, need, need_tokens, on, out, ptr, raw_stream, workspace as _ws

_IO = (torch.float32, torch.bfloat16)
_F32, _BF16 = torch.float32, torch.bfloat16


def _common(a, q, k, v, g, lead, scale):
    """Checks q, k, v, g (``lead`` token dimensions each) and fills sizes, strides and pointers of ``a``;
    returns the device and the tokens' dimensions."""
    try:
        dtype, dev, qs, vs, gs = q.dtype, q.device, q.shape, v.shape, g.shape
        tokens, (Hk, dk), (H, dv) = qs[:lead], qs[lead:], vs[lead:]
        # what a program passes normally: plain contiguous tensors that fit each other
        plain = (q.is_cuda and (dtype is _BF16 or dtype is _F32) and k.dtype is dtype and v.dtype is dtype and g.dtype is _F32
                 and k.shape == qs and vs[:lead] == tokens and (gs == vs[:lead + 1] or gs == (H,))
                 and k.device == dev and v.device == dev and g.device == dev and q.is_contiguous()
                 and k.is_contiguous() and v.is_contiguous() and g.is_contiguous() and type(q) is type(k) is type(v) is type(g) is Tensor)
    except (AttributeError, TypeError, ValueError):
        plain = False
    if not plain:
        tokens, Hk, dk, H, dv = _check(a, q, k, v, g, lead)
        dtype, dev, gs = q.dtype, q.device, g.shape
    if Hk == 0 or H % Hk:
        raise ValueError(f"the {Hk} key heads must divide the {H} value heads")
    if len(gs) == 1:
        a.flags = nat.FV_LA_HEAD_DECAY
    if H >= 1 << 31 or dk >= 1 << 31 or dv >= 1 << 31 or dk == 0:
        raise ValueError(f"{H} heads of {dk} x {dv} channels are out of range")
    a.H, a.Hk, a.dk, a.dv = H, Hk, dk, dv
    a.type = nat.FV_TYPE_F32 if dtype is _F32 else nat.FV_TYPE_BF16
    a.scale = dk**-0.5 if scale is None else scale
    a.q, a.k, a.v, a.g = q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr()
    return dev, tokens


def _check(a, q, k, v, g, lead):
    """The long way: says what is wrong, or finds the token strides."""
    check_tensor("q", q, _IO, contiguous=False)
    dtype, dev = q.dtype, q.device
    check_tensor("v", v, (dtype,), dev, contiguous=False)
    check_tensor("g", g, (_F32,), dev, contiguous=False)
    if q.dim() != lead + 2 or v.dim() != lead + 2:
        raise ValueError(f"q and v must have {lead + 2} dimensions, got {list(q.shape)} and {list(v.shape)}")
    tokens = q.shape[:lead]
    Hk, dk = q.shape[lead:]
    H, dv = v.shape[lead:]
    a.q_stride = need_tokens("q", q, dtype, q.shape, dev, lead)
    a.k_stride = need_tokens("k", k, dtype, q.shape, dev, lead)
    a.v_stride = need_tokens("v", v, dtype, (*tokens, H, dv), dev, lead)
    if g.dim() == 1:
        need("g", g, _F32, (H,), dev)
    else:
        a.g_stride = need_tokens("g", g, _F32, (*tokens, H), dev, lead, 1)
    return tokens, Hk, dk, H, dv


def _sequences(a, q, k, v, g, scale, initial_state, cu_seqlens):
    dev, tokens = _common(a, q, k, v, g, 2 if cu_seqlens is None else 1, scale)
    if cu_seqlens is None:
        a.N, a.T = count("batch", tokens[0]), count("tokens", tokens[1])
    else:
        check_tensor("cu_seqlens", cu_seqlens, (torch.int32,), dev)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be [N+1]")
        a.N, a.T = count("sequences", cu_seqlens.numel() - 1), count("rows", tokens[0])
        a.cu_seqlens = cu_seqlens.data_ptr()
    states = (a.N, a.H, a.dk, a.dv)
    if initial_state is not None:
        a.initial_state = need("initial_state", initial_state, _F32, states, dev)
    return dev, states


def _size(fn, a):
    n = int(fn(byref(a)))
    if n == 0:
        nat.check(nat.lib().fastvim_linattn_validate(byref(a)), "fastvim_linattn_workspace_size")
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
    where = on(dev, stream)
    if where is None:
        return _queue(a, v, states, return_state, y, final_state, workspace, dev)
    with where:
        return _queue(a, v, states, return_state, y, final_state, workspace, dev)


def _queue(a, v, states, return_state, y, final_state, workspace, dev):
    y = out("y", y, v, v.dtype, v.shape, dev)
    a.y = y.data_ptr()
    if return_state or final_state is not None:
        final_state = out("final_state", final_state, None, _F32, states, dev)
        a.final_state = final_state.data_ptr()
    lib = nat.lib()
    ws = _ws(workspace, _size(lib.fastvim_linattn_workspace_size, a) if workspace is None else 0, dev)
    nat.check(lib.fastvim_linattn_forward(byref(a), ws.data_ptr(), ws.numel(), raw_stream(dev)), "fastvim_linattn_forward")
    return y if final_state is None else (y, final_state)


def backward(q, k, v, g, dy, scale=None, initial_state=None, d_final_state=None, cu_seqlens=None, grads=None,
             workspace=None, stream=None) -> dict:
    """Queue the gradient for the upstream gradients dy (of y) and d_final_state (of the final states; None:
    zero) and return {"dq", "dk", "dv", "dg"}, with "d_initial_state" where initial_state is given or the
    grads dict asks for it.  Everything is recomputed from the inputs; no forward workspace is needed.
    Gradients of shared key heads are summed over the value heads, a per-head g's over all tokens."""
    a, r = nat.FvLinattnArgs(), nat.FvLinattnGrads()
    dev, states = _sequences(a, q, k, v, g, scale, initial_state, cu_seqlens)
    a.dy_stride = need_tokens("dy", dy, q.dtype, v.shape, dev, v.dim() - 2)
    r.dy = dy.data_ptr()
    if d_final_state is not None:
        r.d_final_state = need("d_final_state", d_final_state, _F32, states, dev)
    grads = grads or {}
    if initial_state is None and grads.get("d_initial_state") is None:
        states = None  # no gradient of the first states
    where = on(dev, stream)
    if where is None:
        return _queue_backward(a, r, q, k, v, g, states, grads, workspace, dev)
    with where:
        return _queue_backward(a, r, q, k, v, g, states, grads, workspace, dev)


def _queue_backward(a, r, q, k, v, g, states, grads, workspace, dev):
    new = {n: out(n, grads.get(n), t, t.dtype, t.shape, dev) for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g))}
    if states is not None:
        new["d_initial_state"] = out("d_initial_state", grads.get("d_initial_state"), None, _F32, states, dev)
    for n, t in new.items():
        setattr(r, n, ptr(t))
    lib = nat.lib()
    ws = _ws(workspace, _size(lib.fastvim_linattn_backward_workspace_size, a) if workspace is None else 0, dev)
    nat.check(lib.fastvim_linattn_backward(byref(a), byref(r), ws.data_ptr(), ws.numel(), raw_stream(dev)),
              "fastvim_linattn_backward")
    return new


def step(q, k, v, g, state, scale=None, slots=None, y=None, status=None, stream=None):
    """Queue one token of B sequences -- q, k [B,Hk,dk], v [B,H,dv], g [B,H] or [H] -- and return y [B,H,dv];
    ``state`` fp32 [S,H,dk,dv] is updated in place.  Row b uses state slots[b] (int32 [B]; a negative slot
    leaves the row out, its y is zero), or state b without slots.  A slot out of range, or one that an
    earlier row of the call has, is found on the device: the row's y is zero, no state changes for it, and
    ``status`` (an int32 tensor of one element, zeroed by the caller) receives FV_ERR_INDEX."""
    a = nat.FvLinattnStepArgs()
    dev, (B,) = _common(a, q, k, v, g, 1, scale)
    if not isinstance(state, Tensor) or state.dim() != 4:
        check_tensor("state", state, (_F32,), dev)
        raise ValueError(f"state must be [S,H,dk,dv], got {list(state.shape)}")
    S = state.shape[0]
    a.state = need("state", state, _F32, (S, a.H, a.dk, a.dv), dev)
    a.B, a.S = count("rows", B), count("states", S)
    if slots is not None:
        a.slots = need("slots", slots, torch.int32, (B,), dev)
    elif S < B:
        raise ValueError(f"{B} rows need as many states, got {S}")
    if status is not None:
        a.status = need("status", status, torch.int32, (1,), dev)
    where = on(dev, stream)
    if where is None:
        return _queue_step(a, v, y, dev)
    with where:
        return _queue_step(a, v, y, dev)


def _queue_step(a, v, y, dev):
    y = out("y", y, v, v.dtype, v.shape, dev)
    a.y = y.data_ptr()
    status = nat.lib().fastvim_linattn_step(byref(a), raw_stream(dev))
    if status:
        nat.check(status, "fastvim_linattn_step")
    return y
