"""Linear attention on the GPU where its launches overlap, and at decays and values at the edge of their range."""
import pytest

torch = pytest.importorskip("torch")

from op_testlib import assert_within, attention_bound  # noqa: E402
from pooled_selective_scan_b200 import _native as nat  # noqa: E402
from pooled_selective_scan_b200 import linattn, ssm  # noqa: E402
from test_linattn_gpu import check_forward, check_gradient, inputs, reference  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F32, BF16 = torch.float32, torch.bfloat16


def offsets(lengths):
    return torch.tensor([0] + list(lengths), device="cuda").cumsum(0).to(torch.int32)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_packed_calls_in_a_row_on_one_workspace(dtype):
    """Packed calls one behind the other on one workspace: with sequences that are cut, with none to cut (whose
    joining launch has nothing to do), with none but empty ones and with bad offsets (whose launches have nothing
    to do at all).  Each gives what it gives alone."""
    H, Hk, dk, dv = 2, 1, 64, 40
    lengths = [[3000, 700, 64], [1260] * 3, [3764, 0, 0], [0, 0, 0], [5, 3700, 59]]
    rows = 3780
    d = inputs(61, rows, 3, H, Hk, dk, dv, dtype)
    x = [d[n] for n in ("q", "k", "v", "g")]
    cus = [offsets(n) for n in lengths]
    bad = torch.tensor([0, 900, 800, 3780], dtype=torch.int32, device="cuda")
    empty = lambda t: torch.full_like(t, 7.0)  # noqa: E731

    def forward(cu, ws=None):
        return linattn.forward(*x, cu_seqlens=cu, initial_state=d["s0"], y=empty(d["v"]), final_state=empty(d["s0"]), workspace=ws)

    def backward(cu, ws=None):
        grads = {n: empty(d[m]) for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("d_initial_state", "s0"))}
        r = linattn.backward(*x, d["dy"], initial_state=d["s0"], d_final_state=d["ds"], cu_seqlens=cu, grads=grads, workspace=ws)
        return tuple(r[n] for n in sorted(r))

    size = max(f(*x, cu_seqlens=cus[0]) for f in (linattn.workspace_size, linattn.backward_workspace_size))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for call in (forward, backward):
        alone = []
        for cu in cus:
            alone.append(call(cu))
            torch.cuda.synchronize()
        for _ in range(4):
            got = []
            for cu in cus:
                got += [call(cu, ws), call(bad, ws)]
            for i, r in enumerate(got):
                for a, b in zip(r, alone[i // 2]):
                    assert torch.equal(a, b) if i % 2 == 0 else (a == 7.0).all()
        assert ssm.device_status(ws) == nat.FV_ERR_INDEX


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T", [(2, 520), (1, 2700)])
def test_replayed_calls_read_the_states_of_their_own_replay(B, T, dtype):
    """Captured calls, cut along their length or not, replayed one behind the other with other inputs each time:
    a launch that reads what the overlapped one before it writes must not see what lay there."""
    H, dk, dv = 2, 64, 136
    sets = [inputs(70 + i, B * T, B, H, 1, dk, dv, dtype, decay=0.05) for i in range(4)]
    shaped = lambda n, x: x if n in ("s0", "ds") else x.reshape(B, T, *x.shape[1:])  # noqa: E731
    sets = [{n: shaped(n, x) for n, x in d.items()} for d in sets]

    def call(d):
        y, s = linattn.forward(d["q"], d["k"], d["v"], d["g"], initial_state=d["s0"], return_state=True)
        r = linattn.backward(d["q"], d["k"], d["v"], d["g"], d["dy"], initial_state=d["s0"], d_final_state=d["ds"])
        return {**r, "y": y, "s": s}

    want = [call(d) for d in sets]
    now = {n: x.clone() for n, x in sets[0].items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(now)
    got = []
    for _ in range(5):
        for d in sets:
            for n in now:
                now[n].copy_(d[n])
            graph.replay()
            got.append({n: x.clone() for n, x in out.items()})
    for i, r in enumerate(got):
        for n in r:
            assert torch.equal(r[n], want[i % len(sets)][n]), n


# dg of a token is e^g <gradient of the state behind it, state before it>: behind a strong decay a small sum beside
# neighbours of ordinary size, of which nothing may be left in it.  Its bound is therefore relative to its own
# magnitudes: fp32's rounding of some (2 dk + 576) terms (op_testlib), bf16 calls with the three-part operands of
# what feeds dg (2^-25 each) and the accumulators' dropped bits (2^-22 for each of up to 16 steps of a product).
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fall", [-5.0, -10.0, -20.0, -40.0])
@pytest.mark.parametrize("T,dk,dv", [(50, 64, 64), (300, 48, 72), (256, 128, 64)])
def test_decay_gradient_of_single_falls(T, dk, dv, fall, dtype):
    H = 2
    d = inputs(T + dk, T, 1, H, H, dk, dv, dtype, decay=0.01)
    d["g"][3::29] = fall
    r = linattn.backward(*(d[n][None] for n in ("q", "k", "v", "g", "dy")), initial_state=d["s0"], d_final_state=d["ds"])
    ref, big = reference(d, [T], dk**-0.5, True, True)
    bound = attention_bound(ref[3], big[3], F32, F32, dk) + (2.0**-18 * big[3] if dtype == BF16 else 0)
    assert_within(r["dg"][0], ref[3], bound, "dg")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decay_gradient_between_large_states(dtype):
    """A large state enters the falls of a chunk and a large gradient of the state leaves it: dg takes their product
    times the falls, which is of ordinary size where the product alone would leave fp32."""
    T, H, dk, dv = 200, 2, 64, 72
    d = inputs(5, T, 1, H, H, dk, dv, dtype, decay=0.01)
    d["s0"] *= 2.0**70
    d["ds"] *= 2.0**70
    d["g"][3], d["g"][50] = -60.0, -40.0
    r = linattn.backward(*(d[n][None] for n in ("q", "k", "v", "g", "dy")), initial_state=d["s0"], d_final_state=d["ds"])
    ref, big = reference(d, [T], dk**-0.5, True, True)
    bound = attention_bound(ref[3], big[3], F32, F32, dk) + (2.0**-18 * big[3] if dtype == BF16 else 0)
    assert_within(r["dg"][0], ref[3], bound, "dg")


# ---- log decays above 0 ---------------------------------------------------------------------------
# Taken as they are while no run of up to 128 tokens sums to more than 80.  The bounds of the other tests hold: a
# weight e^x with |x| up to 80 has an exponent of base 2 below 128, whose half step 2^-18 is the largest error
# that the weight takes over, and at most four weights meet in a term: 2^-16, where the bound's least (2 dk + 576)
# 2^-24 is above 2^-15.


def rising(kind, T, H):
    gen = torch.Generator(device="cuda").manual_seed(T)
    g = -0.1 * torch.rand(T, H, device="cuda", generator=gen)
    if kind == "fall behind a rise":
        g[0::50], g[1::50] = 30.0, -95.0
    elif kind == "rise behind a fall":
        g[0::50], g[1::50] = -100.0, 35.0
    elif kind == "anywhere between e^-35 and e^35":
        G = 70 * torch.rand(T + 1, H, device="cuda", generator=gen, dtype=torch.float64) - 35
        g = G.diff(dim=0).float()
    elif kind == "small steps both ways":
        g = 0.3 * torch.randn(T, H, device="cuda", generator=gen)
    elif kind == "a slow rise":
        g = (78.0 / 128 * torch.rand(T, H, device="cuda", generator=gen))
        g[100::128] = -60.0
    else:  # a fall that the next tokens take back
        g[10], g[40:80] = -97.0, 2.0
    return g


RISES = ["fall behind a rise", "rise behind a fall", "anywhere between e^-35 and e^35", "small steps both ways", "a slow rise",
         "a fall that the next tokens take back"]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,H,Hk,dk,dv", [(40, 2, 1, 64, 64), (300, 2, 2, 64, 72), (129, 1, 1, 128, 64), (1300, 1, 1, 96, 32)])
@pytest.mark.parametrize("kind", RISES)
def test_log_decays_above_zero(kind, T, H, Hk, dk, dv, dtype):
    d = inputs(T + dk, T, 1, H, Hk, dk, dv, dtype)
    d["g"] = rising(kind, T, H)
    if kind == RISES[-1]:
        # what lies before the fall is all that the outputs have
        d["v"][11:] = 0
        d["s0"].zero_()
    elif kind == "a slow rise" and T > 300:
        d["g"][300:] -= 0.5  # else the state leaves fp32
    x = [d[n][None] for n in ("q", "k", "v", "g")]
    for ask in (True, False):
        r = linattn.forward(*x, initial_state=d["s0"], return_state=ask)
        y, s = r if ask else (r, None)
        check_forward(d, [T], y, s, dk**-0.5, True, dtype)
    r = linattn.backward(*x, d["dy"][None], initial_state=d["s0"], d_final_state=d["ds"])
    check_gradient(d, [T], r, dk**-0.5, True, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_log_decays_above_zero_packed(dtype):
    """Short sequences beside one another: a rise in one takes nothing from the others."""
    lengths, H, dk, dv = [7, 0, 200, 1, 64, 130], 2, 40, 64
    d = inputs(63, sum(lengths), len(lengths), H, 1, dk, dv, dtype)
    d["g"] = torch.cat([rising(RISES[i % 4], n, H) for i, n in enumerate(lengths) if n])
    x = [d[n] for n in ("q", "k", "v", "g")]
    cu = offsets(lengths)
    y, s = linattn.forward(*x, initial_state=d["s0"], cu_seqlens=cu, return_state=True)
    check_forward(d, lengths, y, s, dk**-0.5, True, dtype)
    r = linattn.backward(*x, d["dy"], initial_state=d["s0"], d_final_state=d["ds"], cu_seqlens=cu)
    check_gradient(d, lengths, r, dk**-0.5, True, dtype)


# dg where every token decays alike and strongly, so that the pairs of neighbours carry it: a product of two scores with
# one weight.  Of a term's magnitude, a score of 64 channels is off by at most 4 2^-23 (an accumulator drops what lies
# behind its last bit at each of four steps), twice; its weight by 2^-21 (two powers of at most 2^-22 each); its
# products by 3 2^-24; the sums over pairs and tokens by some 16 2^-24.  Together below 2^-18.6.
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("decay", [-0.5, -1.0, -2.0, -2.7])
def test_decay_gradient_is_as_exact_behind_strong_decays(decay, dtype):
    T, H, dk, dv = 256, 3, 64, 64
    d = inputs(11, T, 1, H, H, dk, dv, dtype)
    d["g"].fill_(decay)
    r = linattn.backward(*(d[n][None] for n in ("q", "k", "v", "g", "dy")), initial_state=d["s0"], d_final_state=d["ds"])
    ref, big = reference(d, [T], dk**-0.5, True, True)
    # And in the 2-norm, where signs are random and errors independent: per term the root mean squares of the same parts
    # (two powers 2^-22.3 together, eight steps of 2^-23 2^-22.3, products and sums 2^-22) are 2^-21.4 of it, and the
    # terms' ratio is the sums'; twice that allows for steps that all drop to one side.
    # (The states' sums have one power a term and no scores.)
    _, state = linattn.forward(*(d[n][None] for n in ("q", "k", "v", "g")), initial_state=d["s0"], return_state=True)
    (_, rs), (_, bs) = reference(d, [T], dk**-0.5, True, False)
    for got, want, most, what in ((r["dg"][0], ref[3], big[3], "dg"), (r["d_initial_state"], ref[4], big[4], "d_initial_state"),
                                  (state, rs, bs, "final state")):
        assert_within(got, want, 2.0**-18.6 * most + 2.0**-100, what)
        assert float((got.double() - want).norm()) <= 2.0**-20.4 * float(want.norm()), what


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("what", ["q", "k", "v", "g", "dy"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_non_finite_values_stay_in_their_chunk(what, value, dtype):
    """One token's value that is not finite: other sequences and the chunks of up to 128 tokens on the side that the
    formulas do not reach keep every bit; in the forward a q reaches its own token alone."""
    lengths, H, dk, dv = [200, 400, 30], 2, 64, 72
    d = inputs(17, sum(lengths), 3, H, 1, dk, dv, dtype)
    cu = offsets(lengths)

    def call():
        x = [d[n] for n in ("q", "k", "v", "g")]
        y, s = linattn.forward(*x, initial_state=d["s0"], cu_seqlens=cu, return_state=True)
        r = linattn.backward(*x, d["dy"], initial_state=d["s0"], d_final_state=d["ds"], cu_seqlens=cu)
        return {**r, "y": y, "s": s}

    clean = call()
    at = 200 + 150
    d[what][at, 0] = value
    got = call()
    chunk = slice(200 + 128, 200 + 256)
    for n, x in got.items():
        if n in ("s", "d_initial_state"):
            same = [0, 2]
        elif what == "dy" and n == "y" or what in ("dy", "q") and n == "s":
            same = range(630)
        elif what == "q" and n == "y":
            same = [i for i in range(630) if i != at]
        else:  # q, dy reach earlier tokens' gradients, k, v later ones', g both
            same = list(range(200)) + list(range(600, 630))
            if n == "y" or what in ("k", "v"):
                same += range(200, chunk.start)
            if n != "y" and what in ("q", "dy"):
                same += range(chunk.stop, 600)
        same = list(same)
        assert torch.equal(x[same], clean[n][same]), n
        assert torch.isfinite(clean[n]).all()
    reached = "y" if what != "dy" else "dk"
    assert not torch.isfinite(got[reached]).all()
