"""Cases of the linear-attention and RMS-norm operators, with their plain forms.

Linear attention with a decay for each head (``linattn``): per sequence and value head, with the
key head of its group, S_t = exp(g_t) S_{t-1} + k_t v_t^T and y_t = scale S_t^T q_t.  ``forward``
takes whole sequences (dense, or packed with ``cu_seqlens``), ``backward`` is its gradient and
``step`` advances kept states by one token.  The RMS norm (``rmsnorm``) adds the residual stream,
normalises and scales, optionally to 8 bits with scales, and has its gradient.

Shapes are those of the pooled-scan workloads: E = 384, 768 or 1536 channels split into heads, token
grids of 14 x 14 (224 px), 64 x 64 (1024 px) and 128 x 128 (2048 px).
"""
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # the smallest prefill: two 224 px images (14 x 14 tokens) of a 384-channel block in the
        # framework's fp32, where launches and latency count
        {"name": "prefill_tiny_f32", "op": "prefill", "type": "f32", "B": 2, "T": 196, "H": 6, "Hk": 6, "dk": 64,
         "dv": 64, "decay": "token", "state": False},
        # odd sizes in fp32: heads that are no power of two, shared keys, a length that ends inside a tile
        {"name": "prefill_odd_f32", "op": "prefill", "type": "f32", "B": 3, "T": 1021, "H": 6, "Hk": 2, "dk": 40,
         "dv": 72, "decay": "token", "state": True},
        # the ordinary call: 16 images at 1024 px (64 x 64 tokens), 768 channels in heads of 64
        {"name": "prefill_grid_bf16", "op": "prefill", "type": "bf16", "B": 16, "T": 4096, "H": 12, "Hk": 12,
         "dk": 64, "dv": 64, "decay": "token", "state": False},
        # serving: packed prompts of very different lengths (some empty, some of one token) that continue
        # kept states; queries and keys shared by all heads, as in state-space models
        {"name": "prefill_ragged_bf16", "op": "prefill", "type": "bf16", "N": 40, "total": 50021, "H": 24, "Hk": 1,
         "dk": 128, "dv": 64, "decay": "token", "state": True},
        # one long sequence (four 128 x 128 grids in a row), few heads: split over its length
        {"name": "prefill_long_bf16", "op": "prefill", "type": "bf16", "B": 1, "T": 65536, "H": 12, "Hk": 12,
         "dk": 128, "dv": 128, "decay": "head", "state": True},
        # training step of the ordinary call
        {"name": "gradient_grid_bf16", "op": "gradient", "type": "bf16", "B": 8, "T": 4096, "H": 12, "Hk": 12,
         "dk": 64, "dv": 64, "decay": "token", "state": False},
        # training on packed sequences in fp32: shared keys, one decay a head, gradients of the states
        {"name": "gradient_ragged_f32", "op": "gradient", "type": "f32", "N": 9, "total": 6007, "H": 6, "Hk": 3,
         "dk": 48, "dv": 64, "decay": "head", "state": True},
        # one token of one sequence: latency
        {"name": "step_one_f32", "op": "step", "type": "f32", "B": 1, "S": 1, "H": 6, "Hk": 6, "dk": 64, "dv": 64,
         "decay": "token", "slots": False},
        # one token of each of 256 sequences whose states are kept in slots of a larger pool
        {"name": "step_many_bf16", "op": "step", "type": "bf16", "B": 256, "S": 288, "H": 12, "Hk": 4, "dk": 128,
         "dv": 128, "decay": "token", "slots": True},
        # four single tokens through a block's norm: latency
        {"name": "norm_few_bf16", "op": "norm", "type": "bf16", "M": 4, "E": 768, "res": "bf16", "out": "bf16",
         "block": 0},
        # 16 images at 1024 px, 1536 channels, fp32 residual stream, output in 8 bits for the next product
        {"name": "norm_grid_fp8", "op": "norm", "type": "bf16", "M": 65536, "E": 1536, "res": "f32", "out": "fp8",
         "block": 128},
        # its training step at 768 channels
        {"name": "norm_gradient_bf16", "op": "norm_gradient", "type": "bf16", "M": 65536, "E": 768, "res": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "gradient", "step", "norm", "norm_gradient"])
    t = rng.choice(["bf16", "bf16", "f32"])
    if op in ("prefill", "gradient"):
        H = _log(rng, 1, 24)
        Hk = rng.choice([h for h in range(1, H + 1) if H % h == 0])
        dk, dv = 8 * rng.randint(2, 16), 8 * rng.randint(2, 16)
        most = {"prefill": 1 << 19, "gradient": 1 << 17}[op] // (4 if t == "f32" else 1)
        total = max(1, min(_log(rng, 1, 65536), most // H))
        c = {"op": op, "type": t, "H": H, "Hk": Hk, "dk": dk, "dv": dv, "decay": rng.choice(["token", "token", "head"]),
             "state": rng.random() < 0.5}
        if rng.random() < 0.4:
            return {**c, "N": _log(rng, 1, 48), "total": total}
        B = _log(rng, 1, max(1, min(16, total)))
        return {**c, "B": B, "T": max(1, total // B)}
    if op == "step":
        B, H = _log(rng, 1, 256), _log(rng, 1, 16)
        return {"op": op, "type": t, "B": B, "S": B + rng.randint(0, 40), "H": H,
                "Hk": rng.choice([h for h in range(1, H + 1) if H % h == 0]), "dk": 8 * rng.randint(2, 16),
                "dv": 8 * rng.randint(2, 16), "decay": rng.choice(["token", "head"]), "slots": rng.random() < 0.5}
    t = rng.choice(["bf16", "f32", "f16"])
    E = 4 * _log(rng, 16, 1024)
    M = max(1, min(_log(rng, 1, 65536), (1 << 26) // E))
    res = rng.choice([t, "f32"])
    if op == "norm_gradient":
        return {"op": op, "type": t, "M": M, "E": E, "res": res}
    out = rng.choice([t, "fp8"])
    if out == "fp8" and rng.random() < 0.5:
        return {"op": op, "type": t, "M": M, "E": 128 * max(1, E // 128), "res": res, "out": out, "block": 128}
    return {"op": op, "type": t, "M": M, "E": E, "res": res, "out": out, "block": 0}


# ---- inputs ------------------------------------------------------------------------------------


def _lengths(N, total, gen):
    """N lengths that sum to total, spread over two orders of magnitude, with an empty and a one-token
    sequence among them where there is room."""
    if N == 1:
        return [total]
    w = torch.exp(4.5 * torch.rand(N, generator=gen, dtype=torch.float64))
    if N > 3:
        w[1] = 0.0
    n = torch.floor(w / w.sum() * total).long()
    if N > 3 and total > 8 * N:
        n[2] = 1
    n[0] += total - int(n.sum())
    return [int(v) for v in n]


def _decay(case, shape, g):
    """Log decays -A_h softplus(n - 3): steps and rates as a state-space block has them; one constant a
    head, 1 - 2^-(3 + 5 h / H), where the case says so."""
    H = case["H"]
    h = torch.arange(H, device="cuda", dtype=torch.float32)
    if case["decay"] == "head":
        return torch.log1p(-torch.exp2(-(3.0 + 5.0 * h / H)))
    A = 1.0 + 15.0 * h / max(1, H - 1)
    n = torch.randn(shape, device="cuda", generator=g)
    return -A * torch.nn.functional.softplus(n - 3.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    rand = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    t = TYPES[case["type"]]
    st = {"case": case}
    if case["op"] in ("prefill", "gradient"):
        H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
        if "N" in case:
            n = _lengths(case["N"], case["total"], torch.Generator().manual_seed(seed))
            st["lengths"] = n
            st["cu"] = torch.tensor([0] + n, device="cuda").cumsum(0).to(torch.int32)
            lead, N = (case["total"],), case["N"]
        else:
            st["lengths"] = st["cu"] = None
            lead, N = (case["B"], case["T"]), case["B"]
        st["q"], st["k"], st["v"] = (rand(*lead, h, d).to(t) for h, d in ((Hk, dk), (Hk, dk), (H, dv)))
        st["g"] = _decay(case, (*lead, H), g)
        st["s0"] = rand(N, H, dk, dv) if case["state"] else None
        if case["op"] == "gradient":
            st["dy"] = rand(*lead, H, dv).to(t)
            st["ds"] = rand(N, H, dk, dv) if case["state"] else None
    elif case["op"] == "step":
        B, H, Hk, dk, dv = case["B"], case["H"], case["Hk"], case["dk"], case["dv"]
        st["q"], st["k"], st["v"] = rand(B, Hk, dk).to(t), rand(B, Hk, dk).to(t), rand(B, H, dv).to(t)
        st["g"] = _decay(case, (B, H), g)
        st["s"] = rand(case["S"] if case["slots"] else B, H, dk, dv)
        st["slots"] = torch.randperm(case["S"], device="cuda", generator=g)[:B].to(torch.int32) if case["slots"] else None
    else:
        M, E, r = case["M"], case["E"], TYPES[case["res"]]
        st["w"] = 1.0 + 0.1 * rand(E)
        if case["op"] == "norm":
            st["x"], st["r"] = rand(M, E).to(t), (3.0 * rand(M, E)).to(r)
        else:
            st["s"], st["dy"], st["ds"] = (3.0 * rand(M, E)).to(r), rand(M, E).to(t), rand(M, E).to(r)
    return st


EPS = 1e-5

# ---- plain forms: chunks of C tokens as batched products, 32 bits ---------------------------------


def _pad(x, lengths):
    """Packed rows [total, ...] as [N, longest, ...] with zeros behind each sequence."""
    n = torch.tensor(lengths, device=x.device)
    at = torch.arange(max(max(lengths), 1), device=x.device)
    keep = at[None, :] < n[:, None]
    row = (torch.cumsum(n, 0) - n)[:, None] + at[None, :]
    y = x[torch.where(keep, row, 0)] if len(x) else x.new_zeros(*keep.shape, *x.shape[1:])
    return torch.where(keep.reshape(*keep.shape, *[1] * (x.dim() - 1)), y, 0), keep


def _chunks(x, H, C):
    """[B, T, heads, ...] as [B, H, chunks, C, ...], heads repeated to H, zeros behind T."""
    x = x.repeat_interleave(H // x.shape[2], 2).transpose(1, 2)
    T = x.shape[2]
    n = -(-T // C)
    y = x.new_zeros(x.shape[0], H, n * C, *x.shape[3:])
    y[:, :, :T] = x
    return y.reshape(x.shape[0], H, n, C, *x.shape[3:])


def _dense(st):
    """q, k, v, g (and dy) as [B, T, heads, ...] in 32 bits; the rows that hold tokens where sequences are packed."""
    case = st["case"]
    names = ["q", "k", "v"] + (["dy"] if "dy" in st else [])
    d = {n: st[n].float() for n in names}
    gr = st["g"].expand(*st["v"].shape[:-1]) if case["decay"] == "head" else st["g"]
    d["g"], keep = gr, None
    if st["lengths"] is not None:
        for n in names:
            d[n], _ = _pad(d[n], st["lengths"])
        d["g"], keep = _pad(gr, st["lengths"])
    return d, keep


def _decays(g, C):
    """Within each chunk: cumulative log decays (64 bits), weights exp(G_i - G_j) for i >= j, and exp(G_i),
    exp(G_last - G_j); across the chunks: the decay from the end of chunk c' to the start of chunk c, whose
    last row is the end of the sequence, and the decay from the sequence's start."""
    G = torch.cumsum(g.double(), -1)
    low = torch.ones(C, C, device=g.device, dtype=torch.bool).tril()
    W = torch.where(low, G[..., :, None] - G[..., None, :], -torch.inf).float().exp()
    end = G[..., -1]
    L = torch.nn.functional.pad(torch.cumsum(end, -1), (1, 0))
    n = end.shape[-1]
    below = torch.ones(n + 1, n, device=g.device, dtype=torch.bool).tril(-1)
    D = torch.where(below, L[..., :, None] - L[..., None, 1:], -torch.inf).float().exp()
    return W, G.float().exp(), (end[..., None] - G).float().exp(), D, L.float().exp(), end.float().exp()


def _states(K, V, D, L, tail, s0):
    """The state entering each chunk and, last, the final one: [B, H, chunks + 1, dk, dv]."""
    loc = (K * tail[..., None]).transpose(-1, -2) @ V
    S = (D @ loc.flatten(-2)).unflatten(-1, loc.shape[-2:])
    return S if s0 is None else S + L[..., None, None] * s0[:, :, None]


def _rows(y, T, keep):
    """[B, H, chunks, C, ...] back to [B, T, H, ...], or to packed rows."""
    y = y.flatten(2, 3)[:, :, :T].transpose(1, 2)
    return y if keep is None else y[keep]


def _prefill(st):
    case = st["case"]
    d, keep = _dense(st)
    T = d["q"].shape[1]
    C = 64 if T <= 4096 else 128
    Q, K, V = (_chunks(d[n], case["H"], C) for n in ("q", "k", "v"))
    W, head, tail, D, L, _ = _decays(_chunks(d["g"], case["H"], C), C)
    S = _states(K, V, D, L, tail, st["s0"])
    scale = case["dk"] ** -0.5
    Y = scale * (((Q @ K.transpose(-1, -2)) * W) @ V + head[..., None] * (Q @ S[:, :, :-1]))
    y = _rows(Y, T, keep).to(TYPES[case["type"]])
    return {"y": y, "state": S[:, :, -1].contiguous()} if case["state"] else {"y": y}


def _gradient(st):
    case = st["case"]
    d, keep = _dense(st)
    T, H, Hk, t = d["q"].shape[1], case["H"], case["Hk"], TYPES[case["type"]]
    C = 64 if T <= 4096 else 128
    Q, K, V, Z = (_chunks(d[n], H, C) for n in ("q", "k", "v", "dy"))
    W, head, tail, D, L, end = _decays(_chunks(d["g"], H, C), C)
    W, head = W * case["dk"] ** -0.5, head * case["dk"] ** -0.5
    S = _states(K, V, D, L, tail, st["s0"])[:, :, :-1]
    # the states' gradients: the same sums with the chunks' order reversed
    loc = (Q * head[..., None]).transpose(-1, -2) @ Z
    n = loc.shape[2]
    back = D[..., 1:n, :].transpose(-1, -2)  # [c, c' - 1]: from the start of chunk c' > c back to the end of chunk c
    dS = (back @ loc[:, :, 1:].flatten(-2)).unflatten(-1, loc.shape[-2:])
    if st["ds"] is not None:
        rest = D[..., -1, :]  # from the end of chunk c to the end of the sequence
        dS = dS + rest[..., None, None] * st["ds"][:, :, None]
    first = loc[:, :, 0] + end[:, :, 0, None, None] * dS[:, :, 0]
    X = Z @ V.transpose(-1, -2)
    A, P = (Q @ K.transpose(-1, -2)) * W, X * W
    inq, ink = head[..., None] * (Z @ S.transpose(-1, -2)), tail[..., None] * (V @ dS.transpose(-1, -2))
    dQ, dK = P @ K + inq, P.transpose(-1, -2) @ Q + ink
    dV = A.transpose(-1, -2) @ Z + tail[..., None] * (K @ dS)
    X = X * A
    out = (ink * K).sum(-1)
    G = X.sum(-1, dtype=torch.float64) - X.sum(-2, dtype=torch.float64) + (inq * Q).sum(-1) - out
    G[..., -1] += out.sum(-1) + end * (dS * S).sum((-1, -2))
    dG = G.flip(-1).cumsum(-1).flip(-1).float()
    dq, dk, dv, dg = (_rows(x, T, keep) for x in (dQ, dK, dV, dG))
    dq, dk = (x.unflatten(-2, (Hk, H // Hk)).sum(-2) for x in (dq, dk))
    r = {"dq": dq.to(t), "dk": dk.to(t), "dv": dv.to(t), "dg": dg}
    if case["decay"] == "head":
        r["dg"] = dg.reshape(-1, H).sum(0, dtype=torch.float64).float()
    if case["state"]:
        r["dstate"] = first
    return r


def _step(st):
    case = st["case"]
    H, rows = case["H"], st["slots"].long() if case["slots"] else slice(None)
    q, k = (st[n].float().repeat_interleave(H // case["Hk"], 1) for n in ("q", "k"))
    a = torch.exp(st["g"]).expand(case["B"], H)
    S = a[..., None, None] * st["s"][rows] + k[..., :, None] * st["v"].float()[..., None, :]
    st["s"][rows] = S
    y = case["dk"] ** -0.5 * (q[..., None, :] @ S)[..., 0, :]
    return {"y": y.to(TYPES[case["type"]]), "state": st["s"]}


def _norm(st):
    case = st["case"]
    s = st["x"].float() + st["r"].float()
    y = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS) * st["w"]
    r = {"s": s.to(TYPES[case["res"]])}
    if case["out"] != "fp8":
        return {**r, "y": y.to(TYPES[case["out"]])}
    y = y.unflatten(-1, (-1, case["block"] or case["E"]))
    scale = (y.abs().amax(-1) / 448.0).clamp_min(2.0**-126)
    return {**r, "y": (y / scale[..., None]).flatten(-2).to(torch.float8_e4m3fn), "scales": scale}


def _norm_gradient(st):
    case = st["case"]
    s, dy = st["s"].float(), st["dy"].float()
    r = torch.rsqrt(s.square().mean(-1, keepdim=True) + EPS)
    c = dy * st["w"]
    d = r * (c - s * (r * r * (c * s).mean(-1, keepdim=True))) + st["ds"].float()
    return {"dx": d.to(TYPES[case["type"]]), "dresidual": d.to(TYPES[case["res"]]), "dweight": (dy * s * r).sum(0)}


def _call(state):
    """The framework's calls."""
    from pooled_selective_scan_b200 import linattn, rmsnorm

    case = state["case"]
    op = case["op"]
    if op == "prefill":
        if case["state"]:
            y, s = linattn.forward(state["q"], state["k"], state["v"], state["g"], initial_state=state["s0"],
                                   cu_seqlens=state["cu"], return_state=True)
            return {"y": y, "state": s}
        return {"y": linattn.forward(state["q"], state["k"], state["v"], state["g"], cu_seqlens=state["cu"])}
    if op == "gradient":
        r = linattn.backward(state["q"], state["k"], state["v"], state["g"], state["dy"], initial_state=state["s0"],
                             d_final_state=state["ds"], cu_seqlens=state["cu"])
        out = {n: r[n] for n in ("dq", "dk", "dv", "dg")}
        if case["state"]:
            out["dstate"] = r["d_initial_state"]
        return out
    if op == "step":
        y = linattn.step(state["q"], state["k"], state["v"], state["g"], state["s"], slots=state["slots"])
        return {"y": y, "state": state["s"]}
    if op == "norm_gradient":
        return rmsnorm.backward(state["s"], state["w"], state["dy"], ds=state["ds"], eps=EPS,
                                x_dtype=TYPES[case["type"]])
    if case["out"] == "fp8":
        y, scales, s = rmsnorm.forward_fp8(state["x"], state["w"], residual=state["r"], eps=EPS, block=case["block"])
        return {"s": s, "y": y, "scales": scales}
    y, s = rmsnorm.forward(state["x"], state["w"], residual=state["r"], eps=EPS)
    return {"s": s, "y": y}


def run(state):
    if own:
        return _call(state)
    return {"prefill": _prefill, "gradient": _gradient, "step": _step, "norm": _norm,
            "norm_gradient": _norm_gradient}[state["case"]["op"]](state)


def work(case):
    op, b = case["op"], SIZE[case["type"]]
    if op in ("norm", "norm_gradient"):
        n, r = case["M"] * case["E"], SIZE[case["res"]]
        if op == "norm_gradient":
            return {"bytes": n * (2 * b + 3 * r) + 8 * case["E"], "flops": 12 * n}
        o = n + 4 * (n // case["block"] if case["block"] else case["M"]) if case["out"] == "fp8" else n * SIZE[case["out"]]
        return {"bytes": n * (b + 2 * r) + o + 4 * case["E"], "flops": 6 * n}
    H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
    if op == "step":
        B = case["B"]
        return {"bytes": B * (b * (2 * Hk * dk + 2 * H * dv) + 8 * H * dk * dv) + (4 * B * H if case["decay"] == "token" else 4 * H),
                "flops": 5 * B * H * dk * dv}
    tok, N = (case["total"], case["N"]) if "N" in case else (case["B"] * case["T"], case["B"])
    gd = 4 * H * (tok if case["decay"] == "token" else 1)
    if op == "prefill":
        return {"bytes": tok * b * (2 * Hk * dk + 2 * H * dv) + gd + (8 * N * H * dk * dv if case["state"] else 0),
                "flops": 4 * tok * H * dk * dv}
    return {"bytes": tok * b * (4 * Hk * dk + 3 * H * dv) + 2 * gd + (12 * N * H * dk * dv if case["state"] else 0),
            "flops": 10 * tok * H * dk * dv}


# ---- the definitions in 64 bits, token by token --------------------------------------------------


def exact(case, seed):
    def attention(case, st):
        H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
        grad = case["op"] == "gradient"
        n = st["lengths"] or [case["T"]] * case["B"]
        N, T, dev = len(n), max(max(n), 1), "cuda"
        start = [sum(n[:i]) for i in range(N)]
        flat = lambda x: x.reshape(-1, *x.shape[-2:]).double()  # noqa: E731
        q, k, v = (flat(st[x]) for x in ("q", "k", "v"))
        q, k = (x.repeat_interleave(H // Hk, 1) for x in (q, k))
        g = (st["g"].expand(*st["v"].shape[:-1]) if case["decay"] == "head" else st["g"]).reshape(-1, H).double()
        a = g.exp()
        zero = torch.zeros(N, H, dk, dv, device=dev, dtype=torch.float64)
        S = zero if st["s0"] is None else st["s0"].double()
        scale = dk**-0.5
        # sequences by falling length: at token t the first live[t] of them are still running
        order = sorted(range(N), key=lambda i: -n[i])
        perm = torch.tensor(order, device=dev)
        first = torch.tensor([start[i] for i in order], device=dev)
        live = [sum(x > t for x in n) for t in range(T)]
        S = S[perm].clone()
        y = torch.zeros(len(v), H, dv, device=dev, dtype=torch.float64)
        if grad:
            z = flat(st["dy"])
            dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for t in range(T):
            m = live[t]
            if not m:
                break
            r = first[:m] + t
            S[:m] = a[r][..., None, None] * S[:m] + k[r][..., :, None] * v[r][..., None, :]
            if grad:
                dq[r] = scale * (S[:m] @ z[r][..., None])[..., 0]
            else:
                y[r] = scale * (q[r][..., None, :] @ S[:m])[..., 0, :]
        lead = st["v"].shape[:-2]
        if not grad:
            out = torch.empty_like(S)
            out[perm] = S
            y = y.reshape(*lead, H, dv)
            return {"y": y, "state": out} if case["state"] else {"y": y}
        dS = (zero if st["ds"] is None else st["ds"].double())[perm].clone()
        last = (dS * S).sum((-1, -2))
        for t in reversed(range(T)):
            m = live[t]
            if not m:
                continue
            r = first[:m] + t
            dS[:m] += scale * q[r][..., :, None] * z[r][..., None, :]
            dk_[r] = (dS[:m] @ v[r][..., None])[..., 0]
            dv_[r] = (k[r][..., None, :] @ dS[:m])[..., 0, :]
            dS[:m] *= a[r][..., None, None]
        c = (q * dq).sum(-1) - (k * dk_).sum(-1)
        dg = torch.zeros_like(c)
        for j, i in enumerate(order):
            part = c[start[i]:start[i] + n[i]]
            dg[start[i]:start[i] + n[i]] = part.flip(0).cumsum(0).flip(0) + last[j]
        fold = lambda x: x.reshape(-1, Hk, H // Hk, dk).sum(2).reshape(*lead, Hk, dk)  # noqa: E731
        r = {"dq": fold(dq), "dk": fold(dk_), "dv": dv_.reshape(*lead, H, dv),
             "dg": dg.sum(0) if case["decay"] == "head" else dg.reshape(*lead, H)}
        if case["state"]:
            r["dstate"] = torch.empty_like(dS)
            r["dstate"][perm] = dS
        return r

    st = prepare(case, seed)
    op = case["op"]
    if op in ("prefill", "gradient"):
        return attention(case, st)
    if op == "step":
        H = case["H"]
        at = list(range(case["B"])) if st["slots"] is None else st["slots"].tolist()
        S = st["s"].double()
        q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
        a = torch.exp(st["g"].double())
        y = torch.empty(case["B"], H, case["dv"], device="cuda", dtype=torch.float64)
        for b, s in enumerate(at):
            for h in range(H):
                kh = h // (H // case["Hk"])
                S[s, h] = (a[b, h] if a.dim() == 2 else a[h]) * S[s, h] + torch.outer(k[b, kh], v[b, h])
                y[b, h] = torch.mv(S[s, h].T, q[b, kh]) / case["dk"] ** 0.5
        return {"y": y, "state": S}
    rows = lambda x: x.double()  # noqa: E731
    w = rows(st["w"])
    if op == "norm":
        s = rows(st["x"]) + rows(st["r"])
        y = w * s / torch.sqrt((s * s).sum(-1, keepdim=True) / case["E"] + EPS)
        if case["out"] != "fp8":
            return {"s": s, "y": y}
        big = y.reshape(case["M"], -1, case["block"] or case["E"]).abs().max(-1).values / 448.0
        return {"s": s, "y": None, "scales": big}
    s, dy = rows(st["s"]), rows(st["dy"])
    inv = 1.0 / torch.sqrt((s * s).sum(-1, keepdim=True) / case["E"] + EPS)
    n = s * inv
    c = w * dy
    d = inv * (c - n * (n * c).sum(-1, keepdim=True) / case["E"]) + rows(st["ds"])
    return {"dx": d, "dresidual": d, "dweight": (n * dy).sum(0)}
