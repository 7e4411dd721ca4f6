"""Linear attention on the GPU against the token-by-token recurrence in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

from op_testlib import assert_within, attention, attention_bound  # noqa: E402
from pooled_selective_scan_b200 import _native as nat  # noqa: E402
from pooled_selective_scan_b200 import linattn, ssm  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

F32, BF16 = torch.float32, torch.bfloat16


def inputs(seed, rows, N, H, Hk, dk, dv, dtype, head_decay=False, decay=0.3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    d = {"q": r(rows, Hk, dk).to(dtype), "k": r(rows, Hk, dk).to(dtype), "v": r(rows, H, dv).to(dtype)}
    d["g"] = -decay * r(H if head_decay else rows * H).abs().reshape((H,) if head_decay else (rows, H))
    d["s0"], d["ds"] = r(N, H, dk, dv), r(N, H, dk, dv)
    d["dy"] = r(rows, H, dv).to(dtype)
    return d


def full_g(d, rows, H):
    return d["g"].expand(rows, H) if d["g"].dim() == 1 else d["g"]


def reference(d, lengths, scale, state, grad):
    rows, H = d["v"].shape[:2]
    args = (d["q"], d["k"], d["v"], full_g(d, rows, H), scale, lengths, d["s0"] if state else None)
    big = [x.abs() if x is not None and i != 3 else x for i, x in enumerate(args[:4])] + [abs(scale), lengths,
                                                                                         d["s0"].abs() if state else None]
    if not grad:
        return attention(*args), attention(*big)
    ds = d["ds"] if state else None
    return attention(*args, d["dy"], ds), attention(*big, d["dy"].abs(), ds.abs() if state else None)


def check_forward(d, lengths, y, s, scale, state, dtype):
    (ry, rs), (by, bs) = reference(d, lengths, scale, state, False)
    dk = d["q"].shape[-1]
    assert_within(y.reshape(ry.shape), ry, attention_bound(ry, by, dtype, dtype, dk), "y")
    if s is not None:
        # a state takes no weighted scores: only the two-part rounding of its terms
        assert_within(s, rs, attention_bound(rs, bs, F32, F32, dk) + (2.0**-16 * bs if dtype == BF16 else 0), "final state")


def check_gradient(d, lengths, r, scale, state, dtype):
    ref, big = reference(d, lengths, scale, state, True)
    dk = d["q"].shape[-1]
    rows, H = d["v"].shape[:2]
    for i, name in enumerate(("dq", "dk", "dv")):
        assert_within(r[name].reshape(ref[i].shape), ref[i], attention_bound(ref[i], big[i], dtype, dtype, dk), name)
    # pairs of scores are multiplied in fp32: dg takes the fp32 bound, and the two-part rounding of states
    rg, bg = ref[3], big[3]
    if d["g"].dim() == 1:
        rg, bg = rg.sum(0), bg.sum(0)
    extra = 2.0**-15 * bg if dtype == BF16 else 0
    assert_within(r["dg"].reshape(rg.shape), rg, attention_bound(rg, bg, F32, F32, dk) + extra, "dg")
    if state:
        extra = 2.0**-16 * big[4] if dtype == BF16 else 0
        assert_within(r["d_initial_state"], ref[4], attention_bound(ref[4], big[4], F32, F32, dk) + extra, "d_initial_state")


SHAPES = [  # lengths, H, Hk, dk, dv
    ([1], 1, 1, 8, 8), ([2, 2], 2, 1, 16, 24), ([63], 2, 2, 64, 64), ([64], 1, 1, 64, 64), ([65], 3, 1, 40, 72),
    ([127, 127], 2, 2, 72, 64), ([128], 2, 1, 128, 128), ([129], 1, 1, 128, 64), ([260], 4, 2, 96, 136),
    ([515], 2, 2, 64, 200), ([1300], 1, 1, 32, 256),  # few heads, over 512 tokens: cut along its length
    ([1090], 2, 1, 120, 48),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("lengths,H,Hk,dk,dv", SHAPES)
def test_dense_forward(lengths, H, Hk, dk, dv, state, dtype):
    B, T = len(lengths), lengths[0]
    d = inputs(T + H, B * T, B, H, Hk, dk, dv, dtype)
    shaped = lambda x: x.reshape(B, T, *x.shape[1:])  # noqa: E731
    y, s = linattn.forward(shaped(d["q"]), shaped(d["k"]), shaped(d["v"]), shaped(d["g"]),
                           initial_state=d["s0"] if state else None, return_state=True)
    check_forward(d, lengths, y, s, dk**-0.5, state, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("lengths,H,Hk,dk,dv", SHAPES)
def test_dense_gradient(lengths, H, Hk, dk, dv, state, dtype):
    B, T = len(lengths), lengths[0]
    d = inputs(T + H + 1, B * T, B, H, Hk, dk, dv, dtype, head_decay=H == 2)
    shaped = lambda x: x.reshape(B, T, *x.shape[1:])  # noqa: E731
    g = d["g"] if d["g"].dim() == 1 else shaped(d["g"])
    r = linattn.backward(shaped(d["q"]), shaped(d["k"]), shaped(d["v"]), g, shaped(d["dy"]), scale=0.7,
                         initial_state=d["s0"] if state else None, d_final_state=d["ds"] if state else None)
    assert set(r) == {"dq", "dk", "dv", "dg"} | ({"d_initial_state"} if state else set())
    check_gradient(d, lengths, r, 0.7, state, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_sequence_of_one_head(dtype):
    """Cut into more pieces than add up their states by themselves; the final state, too."""
    T, dk, dv = 4700, 24, 16
    d = inputs(77, T, 1, 1, 1, dk, dv, dtype, decay=0.02)
    x = [d[n][None] for n in ("q", "k", "v", "g")]
    for state in (True, False):
        y, s = linattn.forward(*x, initial_state=d["s0"] if state else None, return_state=True)
        check_forward(d, [T], y, s, dk**-0.5, state, dtype)
        y2 = linattn.forward(*x, initial_state=d["s0"] if state else None)
        (ry, _), (by, _) = reference(d, [T], dk**-0.5, state, False)
        assert_within(y2.reshape(ry.shape), ry, attention_bound(ry, by, dtype, dtype, dk), "y without a state read back")


def test_padded_batch_without_states():
    """One long and many short packed sequences, fewer heads than SMs, no states."""
    lengths = [1, 1200, 0, 7, 64, 128, 129, 1]
    d = inputs(78, sum(lengths), len(lengths), 2, 1, 128, 40, BF16)
    cu = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    y = linattn.forward(*(d[n] for n in ("q", "k", "v", "g")), cu_seqlens=cu)
    check_forward(d, lengths, y, None, 128**-0.5, False, BF16)


PACKED = [([3, 0, 1, 130, 64], 2, 1, 64, 64), ([0, 0], 1, 1, 16, 8), ([1] * 70, 1, 1, 8, 16), ([700, 0, 45, 650], 2, 2, 128, 72),
          ([257], 3, 1, 24, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tail", [0, 5])
@pytest.mark.parametrize("lengths,H,Hk,dk,dv", PACKED)
def test_packed_forward_and_gradient(lengths, H, Hk, dk, dv, tail, dtype):
    """Packed sequences, empty ones among them.  Rows behind the last one hold NaN: they are not read,
    and the outputs there stay as they were."""
    N, used = len(lengths), sum(lengths)
    rows = used + tail
    d = inputs(rows + N, rows, N, H, Hk, dk, dv, dtype)
    for n in ("q", "k", "v", "g", "dy"):
        d[n][used:] = float("nan")
    cu = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    y = torch.full_like(d["v"], 7.0)
    args = (d["q"], d["k"], d["v"], d["g"])
    ws = torch.empty(linattn.workspace_size(*args, cu_seqlens=cu), dtype=torch.uint8, device="cuda")
    y, s = linattn.forward(*args, initial_state=d["s0"], cu_seqlens=cu, return_state=True, y=y, workspace=ws)
    assert ssm.device_status(ws) == nat.FV_OK
    assert (y[used:] == 7.0).all()
    grads = {n: torch.full_like(d[m], 7.0) for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"))}
    r = linattn.backward(*args, d["dy"], initial_state=d["s0"], d_final_state=d["ds"], cu_seqlens=cu, grads=grads)
    for n in grads:
        assert (r[n][used:] == 7.0).all(), n
        r[n] = r[n][:used]
    d = {n: x[:used] if n not in ("s0", "ds") else x for n, x in d.items()}
    check_forward(d, lengths, y[:used], s, dk**-0.5, True, dtype)
    check_gradient(d, lengths, r, dk**-0.5, True, dtype)


@pytest.mark.parametrize("offsets", [[0, 9, 4, 12], [-1, 3, 6, 12], [0, 5, 10, 13]])
def test_bad_offsets_are_reported_and_write_nothing(offsets):
    d = inputs(1, 12, 3, 2, 1, 64, 64, BF16)
    cu = torch.tensor(offsets, device="cuda", dtype=torch.int32)
    args = (d["q"], d["k"], d["v"], d["g"])
    ws = torch.empty(linattn.workspace_size(*args, cu_seqlens=cu), dtype=torch.uint8, device="cuda")
    y = torch.full_like(d["v"], 7.0)
    linattn.forward(*args, cu_seqlens=cu, y=y, workspace=ws)
    assert ssm.device_status(ws) == nat.FV_ERR_INDEX
    assert (y == 7.0).all()
    ws = torch.empty(linattn.backward_workspace_size(*args, cu_seqlens=cu), dtype=torch.uint8, device="cuda")
    grads = {n: torch.full_like(d[m], 7.0) for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"))}
    linattn.backward(*args, d["dy"], cu_seqlens=cu, grads=grads, workspace=ws)
    assert ssm.device_status(ws) == nat.FV_ERR_INDEX
    assert all((x == 7.0).all() for x in grads.values())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_slices_of_a_fused_projection(dtype):
    """q, k, v and g as column slices of wider tensors give what contiguous copies give, bit for bit."""
    B, T, H, Hk, dk, dv = 2, 150, 4, 2, 40, 24
    gen = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.randn(B, T, 2 * Hk * dk + H * dv + 16, device="cuda", generator=gen).to(dtype)
    q = wide[..., :Hk * dk].unflatten(-1, (Hk, dk))
    k = wide[..., Hk * dk:2 * Hk * dk].unflatten(-1, (Hk, dk))
    v = wide[..., 2 * Hk * dk:2 * Hk * dk + H * dv].unflatten(-1, (H, dv))
    g = -torch.rand(B, T, H + 3, device="cuda", generator=gen)[..., 1:H + 1]
    dy = torch.randn(B, T, H, 2 * dv, device="cuda", generator=gen).to(dtype).flatten(2)[..., :H * dv].unflatten(-1, (H, dv))
    plain = [x.contiguous() for x in (q, k, v, g)]
    assert torch.equal(linattn.forward(q, k, v, g), linattn.forward(*plain))
    a, b = linattn.backward(q, k, v, g, dy), linattn.backward(*plain, dy.contiguous())
    assert all(torch.equal(a[n], b[n]) for n in a)
    assert torch.equal(linattn.forward(q[:, :1], k[:, :1], v[:, :1], g[:, :1]),
                       linattn.forward(*(x[:, :1].contiguous() for x in (q, k, v, g))))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_resets_and_strong_decays(dtype):
    """-inf empties the state; steps of very different sizes in one chunk keep their small differences."""
    T, H, dk, dv = 300, 2, 64, 64
    d = inputs(9, T, 1, H, H, dk, dv, dtype)
    d["g"] = -0.01 * torch.rand(T, H, device="cuda")
    d["g"][::7] = -90.0
    d["g"][13::41, 0] = -float("inf")
    d["g"][40:45, 1] = -1e30
    y, s = linattn.forward(*(d[n][None] for n in ("q", "k", "v", "g")), initial_state=d["s0"], return_state=True)
    check_forward(d, [T], y, s, dk**-0.5, True, dtype)
    r = linattn.backward(*(d[n][None] for n in ("q", "k", "v", "g", "dy")), initial_state=d["s0"], d_final_state=d["ds"])
    # the formula's e^g <dS, S> is 0 at -inf, as here
    check_gradient(d, [T], r, dk**-0.5, True, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradient_against_differences(dtype):
    """The gradient of L = sum dy y + sum ds S in every direction of g and of the first state, by central
    differences of the 64-bit formula (the linear inputs follow from the formula itself)."""
    T, H, dk, dv = 21, 2, 16, 16
    d = inputs(3, T, 1, H, 1, dk, dv, dtype)
    r = linattn.backward(*(d[n][None] for n in ("q", "k", "v", "g", "dy")), initial_state=d["s0"], d_final_state=d["ds"])

    def loss(g, s0, q):
        y, s = attention(q, d["k"], d["v"], g, dk**-0.5, [T], s0)
        return float((y * d["dy"].double()).sum() + (s * d["ds"].double()).sum())

    g, s0, q = d["g"].double(), d["s0"].double(), d["q"].double()
    big = reference(d, [T], dk**-0.5, True, True)[1]
    for t, h in ((0, 0), (7, 1), (20, 0)):
        e = torch.zeros_like(g)
        e[t, h] = 2.0**-10
        diff = (loss(g + e, s0, q) - loss(g - e, s0, q)) / 2.0**-9
        # truncation: e^2 / 6 of a third derivative no larger than the sum of magnitudes
        assert abs(float(r["dg"][0, t, h]) - diff) <= (2.0**-20 + 2.0**-13) * float(big[3][t, h])
    e = torch.zeros_like(s0)
    e[0, 1, 3, 5] = 1.0
    assert abs(float(r["d_initial_state"][0, 1, 3, 5]) - (loss(g, s0 + e, q) - loss(g, s0 - e, q)) / 2) <= 2.0**-13 * float(big[4][0, 1, 3, 5])
    e = torch.zeros_like(q)
    e[11, 0, 2] = 1.0
    assert abs(float(r["dq"][0, 11, 0, 2]) - (loss(g, s0, q + e) - loss(g, s0, q - e)) / 2) <= 2.0**-7 * float(big[0][11, 0, 2])


def test_state_in_place_and_continuation():
    """Two halves with the state handed on (in place) equal the whole within the formula's rounding."""
    T, H, dk, dv = 256, 2, 64, 64
    d = inputs(4, T, 1, H, H, dk, dv, BF16)
    x = [d[n][None] for n in ("q", "k", "v", "g")]
    s = d["s0"].clone()
    y0, s0 = linattn.forward(*(t[:, :100].contiguous() for t in x), initial_state=s, final_state=s)
    assert s0.data_ptr() == s.data_ptr()
    y1, s1 = linattn.forward(*(t[:, 100:].contiguous() for t in x), initial_state=s, final_state=s)
    check_forward(d, [T], torch.cat([y0, y1], 1), s1, dk**-0.5, True, BF16)
    long = inputs(6, 1500, 1, 1, 1, 64, 64, BF16)  # cut along its length
    s = long["s0"].clone()
    y, s1 = linattn.forward(*(long[n][None] for n in ("q", "k", "v", "g")), initial_state=s, final_state=s)
    check_forward(long, [1500], y, s1, 0.125, True, BF16)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_repeatable_bit_for_bit(dtype):
    d = inputs(8, 700, 1, 3, 1, 72, 136, dtype)
    x = [d[n][None] for n in ("q", "k", "v", "g")]
    a, b = linattn.forward(*x), linattn.forward(*x)
    assert torch.equal(a, b)
    a, b = (linattn.backward(*x, d["dy"][None], d_final_state=d["ds"]) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_empty_calls():
    for B, T in ((0, 5), (3, 0)):
        d = inputs(2, B * T, B, 2, 1, 64, 64, F32)
        x = [d[n].reshape(B, T, *d[n].shape[1:]) for n in ("q", "k", "v", "g")]
        y, s = linattn.forward(*x, initial_state=d["s0"], return_state=True)
        assert y.shape == (B, T, 2, 64) and torch.equal(s, d["s0"])
        r = linattn.backward(*x[:3], torch.zeros(2, device="cuda"), d["dy"].reshape(B, T, 2, 64), initial_state=d["s0"],
                             d_final_state=d["ds"])
        assert torch.equal(r["d_initial_state"], d["ds"]) and (r["dg"] == 0).all()


# ---- single tokens -----------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,Hk,dk,dv,head", [(1, 1, 1, 8, 8, False), (3, 4, 2, 64, 64, True), (2, 3, 1, 120, 72, False),
                                               (17, 2, 2, 128, 200, False), (5, 6, 3, 40, 256, True)])
def test_step(B, H, Hk, dk, dv, head, dtype):
    d = inputs(B + dk, B, B, H, Hk, dk, dv, dtype, head_decay=head)
    state = d["s0"].clone()
    y = linattn.step(d["q"], d["k"], d["v"], d["g"], state)
    check_forward(d, [1] * B, y, state, dk**-0.5, True, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_steps_equal_the_prompt_form(dtype):
    """A prompt and then single tokens: the same outputs as the whole sequence at once."""
    T, H, dk, dv = 40, 2, 64, 48
    d = inputs(12, T, 1, H, H, dk, dv, dtype)
    x = [d[n][None] for n in ("q", "k", "v", "g")]
    ys, state = linattn.forward(*(t[:, :30].contiguous() for t in x), return_state=True)
    ys = [ys]
    for t in range(30, T):
        ys.append(linattn.step(*(a[:, t].contiguous() for a in x), state)[:, None])
    check_forward(d, [T], torch.cat(ys, 1), state, dk**-0.5, False, dtype)


def test_step_slots():
    """Slots pick the states; a negative one leaves its row out; one out of range, or one that an earlier
    row has, is reported and changes nothing."""
    B, S, H, dk, dv = 6, 9, 2, 64, 64
    d = inputs(7, B, S, H, 1, dk, dv, F32)
    state = d["s0"].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([4, -1, 0, 8, 2, 7], dtype=torch.int32, device="cuda")
    y = linattn.step(d["q"], d["k"], d["v"], d["g"], state, slots=slots, status=status)
    assert int(status) == nat.FV_OK
    rows = [0, 2, 3, 4, 5]
    at = [int(slots[b]) for b in rows]
    sub = {n: d[n][rows] for n in ("q", "k", "v", "g")} | {"s0": d["s0"][at]}
    check_forward(sub, [1] * len(rows), y[rows], state[at], dk**-0.5, True, F32)
    assert (y[1] == 0).all()
    for s in (1, 3, 5, 6):
        assert torch.equal(state[s], d["s0"][s])
    state = d["s0"].clone()
    slots = torch.tensor([4, 9, 4, 3, -5, 4], dtype=torch.int32, device="cuda")
    y = linattn.step(d["q"], d["k"], d["v"], d["g"], state, slots=slots, status=status)
    assert int(status) == nat.FV_ERR_INDEX
    assert (y[[1, 2, 4, 5]] == 0).all()
    sub = {n: d[n][[0, 3]] for n in ("q", "k", "v", "g")} | {"s0": d["s0"][[4, 3]]}
    check_forward(sub, [1, 1], y[[0, 3]], state[[4, 3]], dk**-0.5, True, F32)


# ---- streams, graphs --------------------------------------------------------------------------------


@pytest.mark.parametrize("T,dtype", [(640, BF16), (1300, BF16), (300, F32), (640, F32)])
def test_another_stream_and_a_captured_call(T, dtype):
    """Whole sequences, and ones in pieces: up to eight (whose two kernels overlap) and more."""
    d = inputs(21, T, 1, 2, 1, 64, 64, dtype)
    x = [d[n][None] for n in ("q", "k", "v", "g")]
    want, grads = linattn.forward(*x), linattn.backward(*x, d["dy"][None])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = linattn.forward(*x, stream=side)
    r = linattn.backward(*x, d["dy"][None], stream=side)
    side.synchronize()
    assert torch.equal(y, want) and all(torch.equal(r[n], grads[n]) for n in r)
    # two graphs, each with buffers of its own, replayed on two streams at once
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = linattn.forward(*x)
            back = linattn.backward(*x, d["dy"][None])
        graphs.append((g, out, back))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, out, back in graphs:
        assert torch.equal(out, want) and all(torch.equal(back[n], grads[n]) for n in back)


def test_calls_in_a_row_on_one_workspace():
    """Calls of different shapes on one stream and one workspace, two kernels of a call overlapping: each
    gives what it gives alone."""
    cases = [(2, 196, 2, 64, 64, F32), (1, 515, 1, 40, 72, F32), (1, 1300, 1, 128, 64, BF16), (2, 130, 2, 64, 64, F32)]
    data, alone = [], []
    for i, (B, T, H, dk, dv, t) in enumerate(cases):
        d = inputs(90 + i, B * T, B, H, H, dk, dv, t)
        x = [d[n].reshape(B, T, *d[n].shape[1:]) for n in ("q", "k", "v", "g")]
        data.append((x, d["s0"]))
        alone.append(linattn.forward(*x, initial_state=d["s0"], return_state=True))
    torch.cuda.synchronize()
    ws = torch.empty(max(linattn.workspace_size(*x) for x, _ in data), dtype=torch.uint8, device="cuda")
    got = [linattn.forward(*x, initial_state=s0, return_state=True, workspace=ws) for _ in range(5) for x, s0 in data]
    for i, (y, s) in enumerate(got):
        assert torch.equal(y, alone[i % len(cases)][0]) and torch.equal(s, alone[i % len(cases)][1])
    assert ssm.device_status(ws) == nat.FV_OK


def test_far_offsets():
    """Rows whose element offsets pass 2^31: a wide token stride puts the last tokens there."""
    T, H, dk, dv = 130, 1, 64, 64
    d = inputs(31, T, 1, H, H, dk, dv, BF16)
    stride = (1 << 24) + 8  # 130 tokens: 4 GiB of bf16
    wide = torch.empty((T - 1) * stride + dk, dtype=BF16, device="cuda")
    q = wide.as_strided((1, T, H, dk), (T * stride, stride, dk, 1))
    q.copy_(d["q"][None])
    y = linattn.forward(q, *(d[n][None] for n in ("k", "v", "g")))
    check_forward(d, [T], y, None, dk**-0.5, False, BF16)


def test_heads_without_channels_are_refused():
    e = torch.empty(2, 5, 3, 0, device="cuda")
    with pytest.raises(ValueError, match="out of range"):
        linattn.forward(e, e, torch.empty(2, 5, 3, 8, device="cuda"), torch.zeros(2, 5, 3, device="cuda"))
    with pytest.raises(Exception, match="(?i)shape"):
        linattn.forward(torch.empty(2, 5, 3, 8, device="cuda"), torch.empty(2, 5, 3, 8, device="cuda"), e,
                        torch.zeros(2, 5, 3, device="cuda"))


# A chunk of up to 64 tokens takes its weighted scores in two bf16 parts: what they leave is at most 2^-17 of
# the magnitude (2^-9 of a half step's 2^-8), that of a state in two parts as much, and the output's half step.
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("lengths,H,Hk,dk,dv", [([1], 1, 1, 64, 64), ([1], 3, 1, 128, 40), ([2], 1, 1, 16, 72), ([5, 5, 5], 2, 1, 64, 128),
                                                ([33], 2, 2, 72, 64), ([64, 64], 1, 1, 128, 128)])
def test_short_sequences_take_scores_in_two_parts(lengths, H, Hk, dk, dv, state):
    def bound(ref, big):
        return (2 * dk + 576) * 2.0**-24 * big + 2.0**-8 * ref.abs() + 2.0**-15 * big + 2.0**-100

    B, T = len(lengths), lengths[0]
    for seed in range(8):
        d = inputs(100 * seed + T, B * T, B, H, Hk, dk, dv, BF16, decay=30.0 if seed == 7 else 0.3)
        x = [d[n].reshape(B, T, *d[n].shape[1:]) for n in ("q", "k", "v", "g")]
        s0, ds = (d["s0"], d["ds"]) if state else (None, None)
        y = linattn.forward(*x, initial_state=s0)
        (ry, _), (by, _) = reference(d, lengths, dk**-0.5, state, False)
        assert_within(y.reshape(ry.shape), ry, bound(ry, by), "y")
        r = linattn.backward(*x, d["dy"].reshape(B, T, H, dv), initial_state=s0, d_final_state=ds)
        ref, big = reference(d, lengths, dk**-0.5, state, True)
        for i, name in enumerate(("dq", "dk", "dv")):
            assert_within(r[name].reshape(ref[i].shape), ref[i], bound(ref[i], big[i]), name)
        assert_within(r["dg"].reshape(ref[3].shape), ref[3], attention_bound(ref[3], big[3], F32, F32, dk) + 2.0**-15 * big[3], "dg")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_cut_sequences_captured_and_in_place(dtype):
    """Packed sequences of which some are cut and some are not, replayed on one workspace; the same states
    read and replaced, dense and packed."""
    lengths = [3000, 0, 700, 5, 64, 1200]
    d = inputs(31, sum(lengths), len(lengths), 2, 2, 64, 64, dtype)
    x = [d[n] for n in ("q", "k", "v", "g")]
    cu = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    y, s = linattn.forward(*x, cu_seqlens=cu, initial_state=d["s0"], return_state=True)
    check_forward(d, lengths, y, s, 64**-0.5, True, dtype)
    ws = torch.empty(linattn.workspace_size(*x, cu), dtype=torch.uint8, device="cuda")
    y2, s2 = torch.zeros_like(y), torch.zeros_like(s)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        linattn.forward(*x, cu_seqlens=cu, initial_state=s2, y=y2, final_state=s2, workspace=ws)
    for _ in range(20):
        y2.zero_()
        s2.copy_(d["s0"])
        graph.replay()
        assert torch.equal(y, y2) and torch.equal(s, s2)
    assert ssm.device_status(ws) == nat.FV_OK
    dense = [z[:4800].reshape(2, 2400, *z.shape[1:]) for z in x]
    want = linattn.forward(*dense, initial_state=d["s0"][:2].contiguous(), return_state=True)
    for _ in range(20):
        st = d["s0"][:2].clone()
        got = linattn.forward(*dense, initial_state=st, final_state=st)
        # the pieces' states are joined by another launch here: the same sums, in the same order
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
