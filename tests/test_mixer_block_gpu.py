"""A block's pre-norm and its linear attention together, as a model runs them: norm with the residual,
projections (torch products), attention, and the way back; a prompt and then single tokens."""
import pytest

torch = pytest.importorskip("torch")

from pooled_selective_scan_b200 import linattn, rmsnorm  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

B, T, E, H, Hk, DK, DV = 2, 150, 128, 4, 2, 32, 32


def weights(gen):
    r = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    return {"norm": 1 + 0.1 * r(E), "q": r(E, Hk * DK) / E**0.5, "k": r(E, Hk * DK) / E**0.5, "v": r(E, H * DV) / E**0.5,
            "g": r(E, H) / E**0.5, "out": r(H * DV, E) / (H * DV) ** 0.5}


def project(y, w):
    split = lambda n, h: (y @ w[n]).unflatten(-1, (h, -1))  # noqa: E731
    return split("q", Hk), split("k", Hk), split("v", H), -torch.nn.functional.softplus(y @ w["g"] - 2)


def plain(x, r, w):
    """The block in 64 bits, token by token."""
    s = x + r
    y = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + 1e-5) * w["norm"]
    q, k, v, g = project(y, w)
    q, k = (t.repeat_interleave(H // Hk, 2) for t in (q, k))
    S = torch.zeros(B, H, DK, DV, device="cuda", dtype=torch.float64)
    out = []
    for t in range(x.shape[1]):
        S = torch.exp(g[:, t])[..., None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        out.append(DK**-0.5 * torch.einsum("bhk,bhkv->bhv", q[:, t], S))
    return torch.stack(out, 1).flatten(2) @ w["out"], s


# fp32 stages (the norm, three products of up to 128 terms, the attention of up to 150 tokens) are each within
# (n terms) 2^-24 < 2^-15 of the magnitudes they add; magnitudes exceed results by less than 2^4 in the
# 2-norm here, and four stages follow each other: 2^-9.
REL = 2.0**-9


def near(got, want, what):
    assert float((got.double() - want).norm() / want.norm()) < REL, what


def test_forward_and_gradient_of_a_block():
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = weights(gen)
    x, r, up = (torch.randn(B, T, E, device="cuda", generator=gen) for _ in range(3))
    y, s = rmsnorm.forward(x, w["norm"], residual=r)
    y.requires_grad_()
    q, k, v, g = project(y, w)
    o = linattn.forward(*(t.detach().contiguous() for t in (q, k, v, g)))
    z = o.flatten(2) @ w["out"]
    leaf = {n: t.double().requires_grad_() for n, t in {"x": x, "r": r, "norm": w["norm"]}.items()}
    w64 = {n: t.double() for n, t in w.items()} | {"norm": leaf["norm"]}
    z64, s64 = plain(leaf["x"], leaf["r"], w64)
    near(z, z64.detach(), "output")
    near(s, s64.detach(), "residual stream")
    # the loss is sum(up z) + sum(up s): s feeds the next block too
    (up.double() * (z64 + s64)).sum().backward()
    dout = (up @ w["out"].T).unflatten(-1, (H, DV)).contiguous()
    d = linattn.backward(*(t.detach().contiguous() for t in (q, k, v, g)), dout)
    torch.autograd.backward([q, k, v, g], [d["dq"], d["dk"], d["dv"], d["dg"]])
    n = rmsnorm.backward(s, w["norm"], y.grad, ds=up)
    near(n["dx"], leaf["x"].grad, "dx")
    near(n["dresidual"], leaf["r"].grad, "dresidual")
    near(n["dweight"], leaf["norm"].grad, "dweight")


def test_prompt_then_single_tokens():
    """A prompt through the attention's chunked form, then tokens one by one on the kept states, in slots."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    w = weights(gen)
    x, r = (torch.randn(B, T, E, device="cuda", generator=gen) for _ in range(2))
    z64, _ = plain(x.double(), r.double(), {n: t.double() for n, t in w.items()})
    y, _ = rmsnorm.forward(x[:, :140].contiguous(), w["norm"], residual=r[:, :140].contiguous())
    o, s = linattn.forward(*(t.contiguous() for t in project(y, w)), return_state=True)
    outs = [o]
    pool = torch.zeros(5, H, DK, DV, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = s
    for t in range(140, T):
        y, _ = rmsnorm.forward(x[:, t].contiguous(), w["norm"], residual=r[:, t].contiguous())
        outs.append(linattn.step(*(p.contiguous() for p in project(y, w)), pool, slots=slots)[:, None])
    near(torch.cat(outs, 1).flatten(2) @ w["out"], z64, "output")
    assert (pool[[0, 2, 4]] == 0).all()


def test_eight_bit_norm_into_the_projections():
    """The 8-bit norm's values and scales, taken back to fp32, through the same block: e4m3 is off by at most
    2^-4 of a value (2^-5 in the 2-norm, whose rounding errors spread over the step), and the projections
    and the attention's products of two such inputs carry it at most fourfold."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    w = weights(gen)
    x, r = (torch.randn(B, T, E, device="cuda", generator=gen) for _ in range(2))
    z64, s64 = plain(x.double(), r.double(), {n: t.double() for n, t in w.items()})
    y8, scales, s = rmsnorm.forward_fp8(x, w["norm"], residual=r, block=128)
    y = (y8.float().unflatten(-1, (-1, 128)) * scales[..., None]).flatten(-2)
    o = linattn.forward(*(t.contiguous() for t in project(y, w)))
    assert float(((o.flatten(2) @ w["out"]).double() - z64).norm() / z64.norm()) < 4 * 2.0**-5
    near(s, s64, "residual stream")
