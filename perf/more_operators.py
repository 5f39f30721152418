"""Timing cases of two more layer operators: the gated linear recurrence (prompts,
single tokens, backward) and the norm of queries and keys per head with the position
rotation (forward, backward).

``listed()`` gives the cases, ``prepare`` makes a case's inputs on the GPU, ``run``
does one pass: the library's calls when ``own`` is true, the same operators in
elementary torch operations otherwise.  ``exact`` computes a case from the operator's
definition in 64 bits.  Bytes in ``work`` count each input read once and each output
written once.
"""
from __future__ import annotations

import math

import torch

own = False

F32, BF16 = "f32", "bf16"
_DT = {F32: torch.float32, BF16: torch.bfloat16}
_SIZE = {F32: 4, BF16: 2}
EPS = 1e-5
EVERY = 64                 # tokens between the states that a training forward keeps for its backward


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # One user's next token on a layer of the Mamba-1 block's inner width: latency alone.
        dict(name="scan step, 1 row", op="step", n=1, slots=8, D=1536, dtype=BF16),
        # The decode batch of the repository's step workloads, 256 sequences scattered in a pool of 320.
        dict(name="scan step, 256 rows", op="step", n=256, slots=320, D=1536, dtype=BF16),
        # A few short prompts of odd lengths arriving together, states from and into pool slots.
        dict(name="scan prompt, short", op="prompt", n=7, T=1021, D=1000, dtype=BF16, packed=True, fused=False),
        # A prefill batch as a server packs it: 16 thousand tokens of nine prompts, input and gates side by
        # side in one projection's output.
        dict(name="scan prompt, packed", op="prompt", n=9, T=16384, D=1536, dtype=BF16, packed=True, fused=True),
        # One long document.
        dict(name="scan prompt, long", op="prompt", n=1, T=65536, D=768, dtype=BF16, packed=False, fused=False),
        # fp32 evaluation of equal-length sequences, neither length nor width a multiple of any tile.
        dict(name="scan prompt, fp32", op="prompt", n=2, T=8190, D=1001, dtype=F32, packed=False, fused=False),
        # The gradient of one training layer: the Mamba-1 block's batch 8, L 2048, with the states its forward kept.
        dict(name="scan backward, training", op="bwd", n=8, T=16384, D=1536, dtype=BF16, packed=False),
        # One user's next token of an attention layer: 16 heads of 128, keys shared by four.
        dict(name="qk, 1 token", op="qk", T=1, H=16, G=4, D=128, R=128, pairs=False, far=32768, fused=True, dtype=BF16),
        # The decode batch, every sequence at a place of its own, cut from the fused projection's rows.
        dict(name="qk, 256 tokens", op="qk", T=256, H=16, G=4, D=128, R=128, pairs=False, far=32768, fused=True, dtype=BF16),
        # A prefill of 16 thousand tokens, as many key heads as query heads.
        dict(name="qk, prompt", op="qk", T=16384, H=16, G=16, D=128, R=128, pairs=False, far=16384, fused=False, dtype=BF16),
        # fp32, an odd head width of which less than half is rotated, far positions, odd length.
        dict(name="qk, fp32 partial", op="qk", T=4095, H=6, G=2, D=80, R=32, pairs=True, far=1000000, fused=False, dtype=F32),
        # The gradient of one training layer, batch 4, L 4096.
        dict(name="qk backward, training", op="qkbwd", T=16384, H=16, G=4, D=128, R=128, pairs=False, far=4096, dtype=BF16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes spread over the ranges the listed cases stand for."""
    op = rng.choice(["step", "prompt", "prompt", "bwd", "bwd", "qk", "qk", "qkbwd"])
    dt = rng.choice([F32, BF16])
    if op in ("step", "prompt", "bwd"):
        D = _log_int(rng, 40, 2560)
        D = D // 8 * 8 if rng.random() < 0.7 else D
        if op == "step":
            n = _log_int(rng, 1, 512)
            return dict(op=op, n=n, slots=n + rng.randrange(64), D=D, dtype=dt)
        n = rng.randrange(1, 12)
        T = _log_int(rng, 1, 16000)
        packed = rng.random() < 0.5
        c = dict(op=op, n=n, T=T if packed else n * max(1, T // n), D=D, dtype=dt, packed=packed)
        return c if op == "bwd" else dict(c, fused=rng.random() < 0.5)
    G = rng.choice([1, 2, 3, 4, 8])
    D = rng.choice([16, 32, 40, 64, 72, 80, 96, 100, 128, 160, 256])
    c = dict(op=op, T=_log_int(rng, 1, 8000), H=G * rng.choice([1, 2, 4]), G=G, D=D, R=D if rng.random() < 0.6 else D // 4 * 2,
             pairs=rng.random() < 0.5, far=_log_int(rng, 8, 1000000), dtype=dt)
    return c if op == "qkbwd" else dict(c, fused=rng.random() < 0.5)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _lengths(case, seed):
    """Lengths that add up to T, uneven where the case is packed (some may be zero)."""
    n, T = case["n"], case["T"]
    if not case["packed"]:
        return [T // n] * n
    g = torch.Generator().manual_seed(seed * 7 + 1)
    cuts = sorted(torch.randint(0, T + 1, (n - 1,), generator=g).tolist())
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, dt = case["op"], _DT[case["dtype"]]
    s = dict(case=case, seed=seed)

    def rn(*shape, sd=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * sd).to(dtype)

    def side_by_side(rows, widths):
        """Columns of one projection's output."""
        return rn(rows, sum(widths)).split(list(widths), 1)

    D = case["D"]
    if op in ("step", "prompt", "bwd"):
        # decay rates from channels that hold thousands of tokens to ones that hold a few
        s["decay"] = torch.exp(torch.empty(D, device=dev).uniform_(math.log(1e-3), math.log(4.0), generator=g))
        s["a_bias"], s["x_bias"] = rn(D, sd=0.5, dtype=torch.float32), rn(D, sd=0.5, dtype=torch.float32)
        names = ("x", "a_gate", "x_gate")
        if op == "step":
            s.update(zip(names, side_by_side(case["n"], (D, D, D))))
            s["slots"] = torch.randperm(case["slots"], generator=g, device=dev)[:case["n"]].int()
            s["pool"] = rn(case["slots"], D, dtype=torch.float32)
            return s
        n, T, lens = case["n"], case["T"], _lengths(case, seed)
        s["lens"] = lens
        cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device=dev)
        s["starts"] = cu
        s["cu"] = cu if case["packed"] else None
        lead = (T,) if case["packed"] else (n, T // n)
        flat = side_by_side(T, (D, D, D)) if case.get("fused") else [rn(T, D) for _ in names]
        s.update(zip(names, (t.unflatten(0, lead) if len(lead) > 1 else t for t in flat)))
        if op == "bwd":
            s.update(dy=rn(*lead, D), h0=rn(n, D, dtype=torch.float32), dh=rn(n, D, dtype=torch.float32))
            s["states"] = _kept(s)
        elif case["packed"]:
            s["slots"] = torch.randperm(n + 3, generator=g, device=dev)[:n].int()
            s["pool"] = rn(n + 3, D, dtype=torch.float32)
        return s
    T, H, G, R = case["T"], case["H"], case["G"], case["R"]
    if case.get("fused"):  # queries, keys and as many values in one projection's row
        q, k, _ = side_by_side(T, (H * D, G * D, G * D))
    else:
        q, k = rn(T, H * D), rn(T, G * D)
    s.update(q=q.unflatten(1, (H, D)), k=k.unflatten(1, (G, D)))
    s["wq"], s["wk"] = 1.0 + 0.3 * rn(D, dtype=torch.float32), 1.0 + 0.3 * rn(D, dtype=torch.float32)
    s["freqs"] = (10000.0 ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R)).float()
    s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device=dev, dtype=torch.int32)
    if op == "qkbwd":
        s.update(dq=rn(T, H, D), dk=rn(T, G, D))
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"step": _step, "prompt": _prompt, "bwd": _bwd, "qk": _qk, "qkbwd": _qkbwd}[op](s)


def _own(op, s):
    import selective_state_space_amd as mb
    if op in ("step", "prompt", "bwd"):
        bias = dict(a_bias=s["a_bias"], x_bias=s["x_bias"])
    if op == "step":
        y, h = mb.mb_gated_scan_step(s["x"], s["a_gate"], s["decay"], s["pool"], s["x_gate"], slots=s["slots"], **bias)
        return {"y": y, "h": h}
    if op == "prompt":
        pool = dict(h0=s["pool"], slots=s["slots"]) if "slots" in s else {}
        y, h = mb.mb_gated_scan(s["x"], s["a_gate"], s["decay"], s["x_gate"], cu_seqlens=s["cu"], **pool, **bias)
        return {"y": y, "h": h}
    if op == "bwd":
        dx, da, di, ddecay, dab, dxb, dh0 = mb.mb_gated_scan_bwd(s["x"], s["a_gate"], s["decay"], s["dy"], s["x_gate"], cu_seqlens=s["cu"],
                                                                 h0=s["h0"], dh_out=s["dh"], states=s["states"], **bias)
        return {"dx": dx, "da_gate": da, "dx_gate": di, "ddecay": ddecay, "da_bias": dab, "dx_bias": dxb, "dh0": dh0}
    how = dict(q_weight=s["wq"], k_weight=s["wk"], interleaved=s["case"]["pairs"], eps=EPS)
    if op == "qk":
        q, k = mb.mb_qk_norm_rope(s["q"], s["k"], s["freqs"], s["positions"], **how)
        return {"q": q, "k": k}
    dq, dk, dwq, dwk = mb.mb_qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["freqs"], s["positions"], **how)
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


# plain forms ---------------------------------------------------------------
def _gates(s, up=torch.Tensor.float):
    """Of every token: the decay gate, the log decay, the input's factor and its gate, in fp32."""
    D = s["case"]["D"]
    sa = torch.sigmoid(up(s["a_gate"]).reshape(-1, D) + up(s["a_bias"]))
    si = torch.sigmoid(up(s["x_gate"]).reshape(-1, D) + up(s["x_bias"]))
    la = -up(s["decay"]) * sa
    return sa, la, torch.sqrt(-torch.expm1(2.0 * la)), si


def _scan(la, b):
    """h_t = exp(la_t) h_{t-1} + b_t over the first axis: by doubling.  Spans' decays are taken of their
    sums of logarithms: a product of many decays close to one would add up their roundings."""
    step = 1
    while step < la.shape[0]:
        b = torch.cat([b[:step], torch.addcmul(b[step:], torch.exp(la[step:]), b[:-step])])
        la = torch.cat([la[:step], la[step:] + la[:-step]])
        step *= 2
    return b


def _nonempty(s):
    """(first tokens, last tokens, indices) of the sequences that have any."""
    cu = s["starts"].long()
    live = torch.tensor([i for i, n in enumerate(s["lens"]) if n], dtype=torch.long, device=cu.device)
    return cu[live], cu[live + 1] - 1, live


def _states(s, la, b, h0):
    """Every token's state."""
    first, _, live = _nonempty(s)
    if h0 is not None:
        b = b.index_add(0, first, torch.exp(la[first]) * h0.to(b.dtype)[live])
    return _scan(la.index_fill(0, first, -math.inf), b)


def _before(s, h, h0):
    """The state that every token starts from."""
    first, _, live = _nonempty(s)
    return torch.cat([h[:1], h[:-1]]).index_copy(0, first, h0.to(h.dtype)[live])


def _kept(s):
    """What a training forward keeps: the state that every 64th token starts from."""
    _, la, beta, si = _gates(s, torch.Tensor.double)
    h0 = s["h0"].double()
    h = _states(s, la, beta * si * s["x"].double().reshape(la.shape), h0)
    return _before(s, h, h0)[::EVERY].float().contiguous()


def _prompt(s):
    _, la, beta, si = _gates(s)
    _, last, live = _nonempty(s)
    rows = s["slots"].long() if "slots" in s else None
    h0 = s["pool"][rows] if rows is not None else None
    h = _states(s, la, beta * si * s["x"].float().reshape(la.shape), h0)
    end = torch.zeros(s["case"]["n"], h.shape[1], device=h.device) if h0 is None else h0
    end = end.index_copy(0, live, h[last])
    if rows is not None:
        s["pool"][rows] = end
    return {"y": h.to(s["x"].dtype).view(s["x"].shape), "h": end if rows is None else s["pool"]}


def _step(s):
    _, la, beta, si = _gates(s)
    rows = s["slots"].long()
    h = torch.exp(la) * s["pool"][rows] + beta * si * s["x"].float()
    s["pool"][rows] = h
    return {"y": h.to(s["x"].dtype), "h": s["pool"]}


def _bwd(s):
    x, dy, dt = s["x"].float().flatten(0, -2), s["dy"].float().flatten(0, -2), s["x"].dtype
    sa, la, beta, si = _gates(s)
    first, last, live = _nonempty(s)
    a, b = torch.exp(la), beta * si * x
    before = _before(s, _states(s, la, b, s["h0"]), s["h0"])
    # from the last token to the first: each takes what the token behind it passes on
    on = torch.cat([la[1:], la[:1]]).index_fill(0, last, -math.inf)
    G = _scan(on.flip(0), dy.index_add(0, last, s["dh"][live]).flip(0)).flip(0)
    dla = G * (a * before - a * a * si * x / beta)
    da, di = dla * la * (1.0 - sa), G * b * (1.0 - si)
    dh0 = s["dh"].index_copy(0, live, a[first] * G[first])
    out = {"dx": G * beta * si, "da_gate": da, "dx_gate": di}
    return {**{k: v.to(dt).view(s["x"].shape) for k, v in out.items()}, "ddecay": -(dla * sa).sum(0), "da_bias": da.sum(0), "dx_bias": di.sum(0),
            "dh0": dh0}


def _angles(s):
    a = s["positions"].double()[:, None] * s["freqs"].double()
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _split(t, c):
    """The two members of every rotated pair, and what is not rotated."""
    R = c["R"]
    if c["pairs"]:
        return t[..., 0:R:2], t[..., 1:R:2], t[..., R:]
    return t[..., :R // 2], t[..., R // 2:R], t[..., R:]


def _join(u, v, rest, c):
    return torch.cat([torch.stack([u, v], -1).flatten(-2) if c["pairs"] else torch.cat([u, v], -1), rest], -1)


def _qk(s):
    c, (cos, sin) = s["case"], _angles(s)

    def one(t, w):
        x = t.float()
        u, v, rest = _split(x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w, c)
        return _join(u * cos - v * sin, u * sin + v * cos, rest, c).to(t.dtype)

    return {"q": one(s["q"], s["wq"]), "k": one(s["k"], s["wk"])}


def _qkbwd(s):
    c, (cos, sin) = s["case"], _angles(s)

    def one(t, w, d):
        x = t.float()
        r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        u, v, rest = _split(d.float(), c)
        e = _join(u * cos + v * sin, v * cos - u * sin, rest, c)
        xh, g = x * r, e * w
        return (r * (g - xh * (g * xh).mean(-1, keepdim=True))).to(t.dtype), (e * xh).sum((0, 1))

    dq, dwq = one(s["q"], s["wq"], s["dq"])
    dk, dwk = one(s["k"], s["wk"], s["dk"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op, e, D = case["op"], _SIZE[case["dtype"]], case["D"]
    if op in ("step", "prompt", "bwd"):
        T, n = case["n"] if op == "step" else case["T"], case["n"]
        if op == "bwd":  # x, both gates, dy in, three gradients out; kept states, h0 and dh_out in, dh0 out
            return dict(bytes=7 * T * D * e + -(-T // EVERY) * D * 4 + 3 * n * D * 4 + 6 * D * 4, flops=60 * T * D)
        has = op == "step" or case["packed"]
        return dict(bytes=4 * T * D * e + (2 if has else 1) * n * D * 4 + 3 * D * 4, flops=30 * T * D)
    m = case["T"] * (case["H"] + case["G"]) * D
    small = 4 * case["T"] + 2 * case["R"] + 8 * D
    if op == "qkbwd":
        return dict(bytes=3 * m * e + small + 8 * D, flops=14 * m)
    return dict(bytes=2 * m * e + small, flops=8 * m)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("qk", "qkbwd"):
        return _exact_qk(s)
    return _exact_scan(s)


def _exact_scan(s):
    """The recurrence token by token, all sequences side by side."""
    c, dev = s["case"], s["x"].device
    op, n, D = c["op"], c["n"], c["D"]
    lens = [1] * n if op == "step" else s["lens"]
    wide = lambda t: t.reshape(-1, D).double()  # noqa: E731
    x, decay = wide(s["x"]), s["decay"].double()
    r = 1.0 / (1.0 + torch.exp(-(wide(s["a_gate"]) + s["a_bias"].double())))
    i = 1.0 / (1.0 + torch.exp(-(wide(s["x_gate"]) + s["x_bias"].double())))
    a = torch.exp(-decay * r)
    one_less = -torch.expm1(-2.0 * decay * r)      # 1 - a^2
    beta = torch.sqrt(one_less)
    start = [sum(lens[:j]) for j in range(n)]
    order = sorted(range(n), key=lambda j: -lens[j])   # longest first: the live ones are a prefix
    at = torch.tensor([start[j] for j in order], device=dev)
    live = [sum(1 for v in lens if v > t) for t in range(max(lens) + 1)]
    pooled = "slots" in s
    rows = s["slots"].long()[order] if pooled else torch.tensor(order, device=dev)
    src = s["pool"] if pooled else s.get("h0")
    h = torch.zeros(n, D, dtype=torch.float64, device=dev) if src is None else src.double()[rows]
    u = beta * i * x
    H, before = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(max(lens)):
        m = live[t]
        j = at[:m] + t
        before[j] = h[:m]
        h[:m] = a[j] * h[:m] + u[j]
        H[j] = h[:m]
    if op != "bwd":
        pool = s["pool"].double() if pooled else torch.empty_like(h)
        pool[rows] = h
        return {"y": H.view(s["x"].shape), "h": pool}
    G, c0 = wide(s["dy"]), s["dh"].double()[rows]
    for t in range(max(lens) - 1, -1, -1):
        m = live[t]
        j = at[:m] + t
        G[j] += c0[:m]
        c0[:m] = a[j] * G[j]
    dh0 = torch.empty_like(c0)
    dh0[rows] = c0
    dlog = G * (before * a) - G * i * x * (1.0 - one_less) / beta
    dr, di = -decay * dlog, G * beta * x
    pre_r, pre_i = dr * r * (1.0 - r), di * i * (1.0 - i)
    out = {"dx": G * beta * i, "da_gate": pre_r, "dx_gate": pre_i}
    return {**{k: v.view(s["x"].shape) for k, v in out.items()}, "ddecay": -torch.einsum("td,td->d", dlog, r), "da_bias": pre_r.sum(0),
            "dx_bias": pre_i.sum(0), "dh0": dh0}


def _exact_qk(s):
    """As complex numbers: a pair times e^(i angle)."""
    c = s["case"]
    R, D = c["R"], c["D"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=s["q"].device), torch.outer(s["positions"].double(), s["freqs"].double()))[:, None]
    j = torch.arange(R // 2, device=s["q"].device)
    lo, hi = (2 * j, 2 * j + 1) if c["pairs"] else (j, j + R // 2)

    def rotated(t, by):
        z = torch.complex(t[..., lo], t[..., hi]) * by
        o = t.clone()
        o[..., lo], o[..., hi] = z.real, z.imag
        return o

    out = {}
    for name, w in (("q", s["wq"]), ("k", s["wk"])):
        x, w = s[name].double(), w.double()
        ms = torch.linalg.vecdot(x, x)[..., None] / D + EPS
        if c["op"] == "qk":
            out[name] = rotated(x / torch.sqrt(ms) * w, turn)
            continue
        e = rotated(s["d" + name].double(), turn.conj())
        dot = torch.einsum("thd,thd,d->th", e, x, w)[..., None] / D
        out["d" + name] = (e * w - x * dot / ms) / torch.sqrt(ms)
        out["dw" + name] = torch.einsum("thd,thd->d", e, x / torch.sqrt(ms))
    return {k: out[k] for k in (("q", "k") if c["op"] == "qk" else ("dq", "dk", "dwq", "dwk"))}
