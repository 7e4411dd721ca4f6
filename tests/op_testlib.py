"""64-bit plain forms of the operators around the layer, token by token, for their tests."""
from __future__ import annotations

import torch


def attention(q, k, v, g, scale, lengths, s0=None, dy=None, ds=None):
    """Packed rows q, k [rows,Hk,dk], v, dy [rows,H,dv], g [rows,H] of sequences of the given lengths, in
    64 bits: (y, final states), or with dy the gradients (dq, dk, dv, dg [rows,H], ds0).  ds: gradient of
    the final states.  Rows behind the last sequence stay zero."""
    H, dv = v.shape[1:]
    Hk, dk = q.shape[1:]
    q, k, v, g = (x.double() for x in (q, k, v, g))
    qh, kh = (x.repeat_interleave(H // Hk, 1) for x in (q, k))
    a = torch.exp(g)
    N = len(lengths)
    S = torch.zeros(N, H, dk, dv, dtype=torch.float64, device=q.device) if s0 is None else s0.double().clone()
    y = torch.zeros_like(v)
    dqh, dkh, dvh, dg = torch.zeros_like(qh), torch.zeros_like(kh), torch.zeros_like(v), torch.zeros_like(g)
    d0 = torch.zeros_like(S)
    start = 0
    for n, T in enumerate(lengths):
        s = S[n].clone()
        states = []
        for t in range(start, start + T):
            if dy is not None:
                states.append(s)
            s = a[t][:, None, None] * s + kh[t][:, :, None] * v[t][:, None, :]
            y[t] = scale * torch.einsum("hk,hkv->hv", qh[t], s)
            if dy is not None:
                dqh[t] = scale * torch.einsum("hkv,hv->hk", s, dy[t].double())
        S[n] = s
        if dy is not None:
            d = torch.zeros_like(s) if ds is None else ds[n].double().clone()
            for t in reversed(range(start, start + T)):
                d = d + scale * qh[t][:, :, None] * dy[t].double()[:, None, :]
                dkh[t] = torch.einsum("hkv,hv->hk", d, v[t])
                dvh[t] = torch.einsum("hkv,hk->hv", d, kh[t])
                before = states[t - start]
                dg[t] = (d * (a[t][:, None, None] * before)).sum((-1, -2))
                d = a[t][:, None, None] * d
            d0[n] = d
        start += T
    if dy is None:
        return y, S
    fold = lambda x: x.reshape(x.shape[0], Hk, H // Hk, dk).sum(2)  # noqa: E731
    return fold(dqh), fold(dkh), dvh, dg, d0


# How far an output may be from its 64-bit value.  `big` is the same formula of the absolute values: the
# sum of the magnitudes of everything that is added.  An fp32 sum of n terms is within n 2^-24 of it; n is
# dk terms of a score, up to 256 of a row of weighted scores, as many of a state, and 64 more for the
# decays (each product of weights is within a few 2^-22).  bf16 inputs are multiplied exactly, but weighted
# scores, or the weighted v of a state nobody reads, are rounded to bf16 once (2^-9 of the magnitude; a pair
# goes one way or the other), and states to two bf16 parts (2^-17).  The result
# is rounded to its own type: half a step.  Weights below 2^-126 are zero (2^-100 covers their products).
def attention_bound(ref, big, dtype, out_dtype, dk):
    n = 2 * dk + 512 + 64
    b = n * 2.0**-24 * big + torch.finfo(out_dtype).eps / 2 * ref.abs() + 2.0**-100
    if dtype == torch.bfloat16:
        b = b + (2.0**-9 + 2.0**-16) * big
    return b


def assert_within(got, ref, bound, what):
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - bound
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{what}: {int((over > 0).sum())}/{over.numel()} outside, worst by {worst:.3e}"
