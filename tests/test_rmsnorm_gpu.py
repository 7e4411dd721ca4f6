"""The RMS norm on the GPU against its formula in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

from op_testlib import assert_within  # noqa: E402
from pooled_selective_scan_b200 import rmsnorm  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5
# E: below a warp's vectors, at and past every group size, odd vector counts, multiples of 4 only
WIDTHS = [4, 8, 20, 128, 252, 256, 384, 516, 768, 1032, 1536, 2048, 2052, 4096, 8192, 12288, 16384]


def data(seed, M, E, t, res):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    return r(M, E).to(t), (2 * r(M, E)).to(res) if res else None, 1 + 0.2 * r(E), r(M, E).to(t), r(M, E).to(res or t)


def norm64(x, r, w):
    s = x.double() + (r.double() if r is not None else 0)
    rstd = torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS)
    return s, s * rstd * w.double(), rstd


# fp32 arithmetic: s is one rounding; the mean of E squares is within E 2^-24, half of that in rstd, and a
# few operations follow (8 2^-24); then the type's own half step.
def y_bound(y, E, t):
    return ((E / 2 + 8) * 2.0**-24 + torch.finfo(t).eps / 2) * y.abs() + 1e-30 + (2.0**-25 if t == F16 else 0)


@pytest.mark.parametrize("t,res", [(F32, None), (F32, F32), (BF16, None), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("E", WIDTHS)
def test_forward(E, t, res):
    x, r, w, _, _ = data(E, 5, E, t, res)
    s64, y64, _ = norm64(x, r, w)
    out = rmsnorm.forward(x, w, residual=r, eps=EPS)
    y = out if r is None else out[0]
    assert_within(y, y64, y_bound(y64, E, t), "y")
    if r is not None:
        assert_within(out[1], s64, (2.0**-24 + torch.finfo(res).eps / 2) * s64.abs() + 2.0**-25, "s")


@pytest.mark.parametrize("t,res", [(F32, F32), (BF16, F32), (F16, None)])
@pytest.mark.parametrize("E,block", [(128, 128), (384, 128), (1536, 128), (4096, 128), (16384, 128), (4, 0), (20, 0), (768, 0),
                                     (1032, 0), (12288, 0)])
def test_forward_fp8(E, block, t, res):
    x, r, w, _, _ = data(E + 1, 6, E, t, res)
    x[2] *= 1e-3
    if res:
        r[2] *= 1e-3
    _, y64, _ = norm64(x, r, w)
    out = rmsnorm.forward_fp8(x, w, residual=r, eps=EPS, block=block)
    y, scales = out[:2]
    assert y.dtype == torch.float8_e4m3fn and y.shape == x.shape
    blocks = y64.unflatten(-1, (-1, block or E))
    big = blocks.abs().amax(-1) / 448
    assert_within(scales.reshape(big.shape), big, (E / 2 + 10) * 2.0**-24 * big, "scales")
    # e4m3: half a step is 2^-4 of the value, 2^-10 of the scale below its normal range (2^-6)
    got = (y.double().unflatten(-1, (-1, block or E)) * scales.double().reshape(big.shape)[..., None])
    assert_within(got, blocks, (2.0**-4 + 2.0**-9) * blocks.abs() + 2.0**-9 * big[..., None], "y")


@pytest.mark.parametrize("t,res", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("M,E", [(1, 4), (3, 20), (1000, 128), (7, 384), (1300, 516), (9, 768), (33, 1032), (700, 1536), (5, 2052),
                                 (6, 4096), (3, 8192), (2, 12288), (4, 16384)])
def test_gradient(M, E, t, res):
    x, r, w, dy, ds = data(M + E, M, E, t, res)
    s = x.to(res) + r if res == t else x.float() + r
    s64, d64, w64 = s.double(), dy.double(), w.double()
    rstd = torch.rsqrt(s64.square().mean(-1, keepdim=True) + EPS)
    n, c = s64 * rstd, d64 * w64
    ref = rstd * (c - n * (n * c).mean(-1, keepdim=True)) + ds.double()
    big = rstd * (c.abs() + n.abs() * (n * c).abs().mean(-1, keepdim=True)) + ds.double().abs()
    out = rmsnorm.backward(s, w, dy, ds=ds, eps=EPS)
    tol = (2 * E + 16) * 2.0**-24 * big
    assert_within(out["dx"], ref, tol + torch.finfo(t).eps / 2 * ref.abs() + 2.0**-25, "dx")
    assert out["dresidual"].dtype == s.dtype
    assert_within(out["dresidual"], ref, tol + torch.finfo(res).eps / 2 * ref.abs() + 2.0**-25, "dresidual")
    assert_within(out["dweight"], (n * d64).sum(0), (M + E / 2 + 16) * 2.0**-24 * (n * d64).abs().sum(0) + 1e-30, "dweight")
    again = rmsnorm.backward(s, w, dy, ds=ds, eps=EPS)
    assert all(torch.equal(out[k], again[k]) for k in out)
    without = rmsnorm.backward(s, w, dy, eps=EPS)["dx"]
    assert_within(without, ref - ds.double(), tol + torch.finfo(t).eps / 2 * (ref - ds.double()).abs() + 2.0**-25, "dx without ds")


def test_gradient_against_differences():
    x, _, w, dy, _ = data(2, 3, 12, F32, None)
    out = rmsnorm.backward(x, w, dy, eps=EPS)
    loss = lambda x, w: float((norm64(x, None, w)[1] * dy.double()).sum())  # noqa: E731
    e = 2.0**-10
    for i in (0, 5, 11):
        d = torch.zeros(3, 12, device="cuda", dtype=torch.float64)
        d[1, i] = e
        diff = (loss(x.double() + d, w) - loss(x.double() - d, w)) / (2 * e)
        assert abs(float(out["dx"][1, i]) - diff) <= 1e-4 * float(dy.abs().max())
        d = torch.zeros(12, device="cuda", dtype=torch.float64)
        d[i] = e
        diff = (loss(x, w.double() + d) - loss(x, w.double() - d)) / (2 * e)
        assert abs(float(out["dweight"][i]) - diff) <= 1e-5 * float(dy.abs().sum())


@pytest.mark.parametrize("t", [F32, BF16])
@pytest.mark.parametrize("E,wide", [(768, 1600), (20, 36)])
def test_rows_of_a_wider_tensor_and_in_place_stream(t, E, wide):
    big, _, w, _, _ = data(4, 10, wide, t, None)
    w = w[:E].contiguous()
    x = big.reshape(2, 5, wide)[..., 8:8 + E] if E != 20 else big.reshape(2, 5, wide)[..., :E]
    r = torch.randn(2, 5, E, device="cuda")
    y, s = rmsnorm.forward(x.contiguous(), w, residual=r, eps=EPS)
    keep = r.clone()
    y2, s2 = rmsnorm.forward(x, w, residual=keep, residual_out=keep, eps=EPS)
    assert s2.data_ptr() == keep.data_ptr()
    assert torch.equal(y, y2) and torch.equal(s, s2)


def test_zero_rows_large_rows_and_non_finite_rows():
    x = torch.zeros(5, 256, device="cuda")
    w = torch.ones(256, device="cuda")
    x[1] = 1e15
    x[2, 3] = float("nan")
    x[3, 200] = float("inf")
    x[4] = 1e-30
    y = rmsnorm.forward(x, w, eps=EPS)
    assert (y[0] == 0).all() and torch.allclose(y[1], torch.ones_like(y[1]), rtol=1e-6)
    assert torch.isnan(y[2]).all() and torch.isnan(y[3, 200]) and (y[4] >= 0).all()
    q, scales = rmsnorm.forward_fp8(x, w, eps=EPS)
    assert (q[0].float() == 0).all() and (scales[0] == 2.0**-126).all()
    assert torch.isnan(scales[2]).all() and torch.isnan(q[2].float()).all()
    assert torch.isnan(scales[3, 1]) and torch.isnan(q[3, 128:].float()).all() and (q[3, :128].float() == 0).all()


def test_no_rows():
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, device="cuda")
    assert rmsnorm.forward(x, w).shape == (0, 64)
    out = rmsnorm.backward(x, w, x)
    assert (out["dweight"] == 0).all() and out["dx"].shape == (0, 64)


def test_another_stream_and_a_captured_call():
    x, r, w, dy, ds = data(8, 300, 768, BF16, F32)
    y, s = rmsnorm.forward(x, w, residual=r)
    g = rmsnorm.backward(s, w, dy, ds=ds)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, s2 = rmsnorm.forward(x, w, residual=r, stream=side)
    g2 = rmsnorm.backward(s2, w, dy, ds=ds, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, s3 = rmsnorm.forward(x, w, residual=r)
        g3 = rmsnorm.backward(s3, w, dy, ds=ds)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y3) and all(torch.equal(g[k], g3[k]) for k in g)


@pytest.mark.parametrize("t", [F32, BF16])
def test_gradient_into_given_buffers(t):
    g = torch.Generator(device="cuda").manual_seed(3)
    s, dy = (torch.randn(37, 200, generator=g, device="cuda").to(t) for _ in range(2))
    w = torch.randn(200, generator=g, device="cuda")
    want = rmsnorm.backward(s, w, dy)
    given = {"dx": torch.empty_like(dy), "dresidual": torch.full_like(s, float("nan")), "dweight": torch.empty_like(w)}
    got = rmsnorm.backward(s, w, dy, grads=given)
    for n in given:
        assert got[n] is given[n] and torch.equal(got[n], want[n])
    one = torch.empty_like(dy)
    got = rmsnorm.backward(s, w, dy, grads={"dx": one, "dresidual": one})
    assert got["dx"] is one and got["dresidual"] is one and torch.equal(one, want["dx"])
