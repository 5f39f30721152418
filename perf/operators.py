"""Timing cases of the layer operators around the scans: linear attention with one
decay per head (prompts, single tokens, backward), the root-mean-square norm with
the residual's addition (also with 8-bit output, and its backward) and the global
gradient norm with clipping.

``listed()`` gives the cases, ``prepare`` makes a case's inputs on the GPU,
``run`` does one pass: the library's calls when ``own`` is true, the same operators
in elementary torch operations otherwise.  ``exact`` computes a case from the
operator's definition in 64 bits.  Bytes in ``work`` count each input read once and
each output written once.
"""
from __future__ import annotations

import math

import torch

own = False

F32, BF16 = "f32", "bf16"
_DT = {F32: torch.float32, BF16: torch.bfloat16}
_SIZE = {F32: 4, BF16: 2}
EPS = 1e-5
FP8_MAX = 448.0            # largest finite e4m3 value
AMAX_MIN = 2.0 ** -96      # amax below this counts as this: a group of zeros keeps a finite scale
CHUNK = 64


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # One user's next token on one layer of the Mamba-3 MIMO block's head shape (16 heads,
        # state 128 x 64): the smallest serving call, latency alone.
        dict(name="attn step, 1 row", op="step", n=1, slots=8, H=16, G=16, Dk=128, Dv=64, dtype=BF16),
        # The decode batch of the repository's step workloads, 256 sequences whose states lie
        # scattered in a pool of 320 (sequences that paused keep theirs).
        dict(name="attn step, 256 rows", op="step", n=256, slots=320, H=16, G=16, Dk=128, Dv=64, dtype=BF16),
        # A few short prompts of odd lengths arriving together, states into pool slots; keys and
        # values shared by pairs of heads.
        dict(name="attn prompt, short", op="prompt", n=7, T=1021, H=8, G=4, Dk=64, Dv=64, dtype=BF16, packed=True),
        # A prefill batch as a server packs it: 16 thousand tokens of nine prompts.
        dict(name="attn prompt, packed", op="prompt", n=9, T=16384, H=16, G=16, Dk=128, Dv=64, dtype=BF16, packed=True),
        # fp32 evaluation of equal-length sequences, length not a multiple of any tile.
        dict(name="attn prompt, fp32", op="prompt", n=2, T=8190, H=16, G=16, Dk=64, Dv=64, dtype=F32, packed=False),
        # The gradient of one training layer: batch 4, L 4096 on the same heads.
        dict(name="attn backward, training", op="bwd", n=4, T=16384, H=16, G=16, Dk=128, Dv=64, dtype=BF16, packed=False),
        # The norm in front of a block for a handful of decoding users, fp32 residual stream.
        dict(name="norm, 4 rows", op="norm", rows=4, D=768, dtype=BF16, res=F32, stride=768),
        # An odd width, rows cut out of a wider buffer so that no row is 16-byte aligned.
        dict(name="norm, odd rows", op="norm", rows=4097, D=1001, dtype=F32, res=F32, stride=1003),
        # The norm before an 8-bit projection, prompt-sized, a scale for every 128 columns.
        dict(name="norm to 8 bits", op="fp8", rows=16384, D=2048, dtype=BF16, res=BF16, group=128),
        # The norm's gradient at the Mamba-1 block's inner width, batch 8 x L 2048.
        dict(name="norm backward", op="nbwd", rows=16384, D=1536, dtype=BF16, res=F32),
        # Clipping the gradients of a two-layer test model: few, small, odd tensors.
        dict(name="clip, small", op="clip", layers=2, d=96, vocab=251, dtype=F32, clipped=True),
        # Clipping the bf16 gradients of a 24-layer model of width 768 with its embedding.
        dict(name="clip, 24 layers", op="clip", layers=24, d=768, vocab=50280, dtype=BF16, clipped=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes spread over the ranges the listed cases stand for."""
    op = rng.choice(["step", "prompt", "prompt", "bwd", "norm", "fp8", "nbwd", "clip"])
    dt = rng.choice([F32, BF16])
    if op in ("step", "prompt", "bwd"):
        H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24])
        G = rng.choice([g for g in (1, 2, 3, 4, 6, 8, 12, 16, 24) if H % g == 0 and g >= H // 4])
        Dk, Dv = rng.choice([16, 24, 40, 64, 80, 96, 128]), rng.choice([16, 20, 32, 64, 96, 128])
        if op == "step":
            n = _log_int(rng, 1, 192)
            return dict(op=op, n=n, slots=n + rng.randrange(64), H=H, G=G, Dk=Dk, Dv=Dv, dtype=dt)
        n = rng.randrange(1, 10)
        T = _log_int(rng, 1, 8000)
        packed = rng.random() < 0.5
        return dict(op=op, n=n, T=T if packed else n * max(1, T // n), H=H, G=G, Dk=Dk, Dv=Dv, dtype=dt, packed=packed)
    if op == "clip":
        d = 8 * rng.randrange(4, 97) + rng.choice([0, 0, 1])
        return dict(op=op, layers=rng.randrange(1, 25), d=d, vocab=_log_int(rng, 200, 50000), dtype=dt, clipped=rng.random() < 0.7)
    rows, D = _log_int(rng, 1, 16384), _log_int(rng, 33, 2048)
    res = rng.choice([F32, dt])
    if op == "norm":
        return dict(op=op, rows=rows, D=D, dtype=dt, res=res, stride=D + rng.choice([0, 0, 1, 8, 64]))
    if op == "fp8":
        return dict(op=op, rows=rows, D=D, dtype=dt, res=res, group=rng.choice([0, 32, 64, 128]))
    return dict(op=op, rows=rows, D=D, dtype=dt, res=res)


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


def _slopes(H, dev):
    """Log decay of head h: -2^(-8 (h + 1) / H), from fast to slow heads."""
    return -torch.exp2(-8.0 * torch.arange(1, H + 1, device=dev, dtype=torch.float64) / H).float()


def _clip_shapes(case):
    """Parameter shapes of a stack of scan blocks: projections, conv, per-channel vectors, embedding."""
    d, e = case["d"], 2 * case["d"]
    layer = [(d,), (e, d), (e, d), (e, 4), (e,), (d // 16 + 32, e), (e, d // 16 or 1), (e,), (e, 16), (e,), (d, e)]
    return [(case["vocab"], d)] + layer * case["layers"] + [(d,)]


def _flat(tensors, dtype):
    """One zeroed buffer and views of it shaped like the tensors, each on a 64-element border."""
    ends = []
    for t in tensors:
        ends.append((ends[-1] if ends else 0) + -(-t.numel() // 64) * 64)
    flat = torch.zeros(ends[-1], dtype=dtype, device=tensors[0].device)
    return flat, [flat[e - -(-t.numel() // 64) * 64:][:t.numel()].view(t.shape) for t, e in zip(tensors, ends)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, dt = case["op"], _DT[case["dtype"]]
    s = dict(case=case, seed=seed)

    def rn(*shape, sd=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * sd).to(dtype)

    if op in ("step", "prompt", "bwd"):
        H, G, Dk, Dv = (case[k] for k in ("H", "G", "Dk", "Dv"))
        s["log_decay"], s["scale"] = _slopes(H, dev), Dk ** -0.5
        if op == "step":
            n = case["n"]
            # one fused projection's row per token, as a layer has it: q | k | v side by side
            qkv = rn(n, H * Dk + G * (Dk + Dv))
            q, k, v = qkv.split([H * Dk, G * Dk, G * Dv], dim=1)
            s.update(q=q.unflatten(1, (H, Dk)), k=k.unflatten(1, (G, Dk)), v=v.unflatten(1, (G, Dv)))
            s["slots"] = torch.randperm(case["slots"], generator=g, device=dev)[:n].int()
            s["pool"] = rn(case["slots"], H, Dk, Dv, dtype=torch.float32)
            return s
        n, lens = case["n"], _lengths(case, seed)
        lead = (case["T"],) if case["packed"] else (n, case["T"] // n)
        s.update(q=rn(*lead, H, Dk), k=rn(*lead, G, Dk), v=rn(*lead, G, Dv), lens=lens)
        cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device=dev)
        s["cu"] = cu if case["packed"] else None
        if op == "bwd":
            s.update(do=rn(*lead, H, Dv), h0=rn(n, H, Dk, Dv, dtype=torch.float32), dh=rn(n, H, Dk, Dv, dtype=torch.float32))
        elif case["packed"]:  # prompts continue from, and leave their state in, pool slots
            s["slots"] = torch.randperm(n + 3, generator=g, device=dev)[:n].int()
            s["pool"] = rn(n + 3, H, Dk, Dv, dtype=torch.float32)
        else:
            s["h0"] = None
        return s
    if op == "clip":
        shapes = _clip_shapes(case)
        s["grads"] = [rn(*sh, sd=2e-3 * (1 + (i % 5))) for i, sh in enumerate(shapes)]
        s["flat"], s["out"] = _flat(s["grads"], dt)  # the clipped gradients land in an optimizer's flat buffer
        s["max_norm"] = 1.0 if case["clipped"] else 1e4
        return s
    rows, D, rdt = case["rows"], case["D"], _DT[case["res"]]
    s["weight"] = 1.0 + 0.3 * rn(D, dtype=torch.float32)
    if op == "nbwd":
        s.update(dy=rn(rows, D), r=rn(rows, D, sd=2.0, dtype=rdt), dr=rn(rows, D, dtype=rdt))
        s["rstd"] = (s["r"].double().square().mean(1) + EPS).rsqrt().float()
        return s
    wide = case.get("stride", D)
    s.update(x=rn(rows, wide)[:, :D], residual=rn(rows, D, sd=2.0, dtype=rdt))
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"step": _step, "prompt": _prompt, "bwd": _bwd, "norm": _norm, "fp8": _fp8, "nbwd": _nbwd, "clip": _clip}[op](s)


def _own(op, s):
    import selective_state_space_amd as mb
    c = s["case"]
    if op == "step":
        o, h = mb.mb_linear_attn_step(s["q"], s["k"], s["v"], s["log_decay"], s["pool"], scale=s["scale"], slots=s["slots"])
        return {"o": o, "h": h}
    if op == "prompt":
        if c["packed"]:
            o, h = mb.mb_linear_attn(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"], cu_seqlens=s["cu"], h0=s["pool"], slots=s["slots"])
        else:
            o, h = mb.mb_linear_attn(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"])
        return {"o": o, "h": h}
    if op == "bwd":
        dq, dk, dv, dh0 = mb.mb_linear_attn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], scale=s["scale"], cu_seqlens=s["cu"],
                                                h0=s["h0"], dh_out=s["dh"])
        return {"dq": dq, "dk": dk, "dv": dv, "dh0": dh0}
    if op == "norm":
        y, r, rstd = mb.mb_rms_norm(s["x"], s["weight"], s["residual"], eps=EPS)
        return {"y": y, "r": r, "rstd": rstd}
    if op == "fp8":
        q, scales, r, rstd = mb.mb_rms_norm_fp8(s["x"], s["weight"], s["residual"], group=c["group"], eps=EPS)
        return {"q": q, "scales": scales, "r": r, "rstd": rstd}
    if op == "nbwd":
        dx, dr, dw = mb.mb_rms_norm_bwd(s["dy"], s["r"], s["rstd"], s["weight"], s["dr"])
        return {"dx": dx, "dr": dr, "dw": dw}
    _, norm = mb.mb_grad_norm_clip(s["grads"], s["max_norm"], out=s["out"])
    return {"norm": norm, "clipped": s["flat"]}


# plain forms ---------------------------------------------------------------
def _rep(t, H):
    return t.repeat_interleave(H // t.shape[-2], -2) if t.shape[-2] != H else t


def _powers(log_decay, e):
    """decay^e for whole exponents e >= 0 (others give 0), shape (H, *e.shape); far positions
    need the exponent in 64 bits."""
    w = torch.exp(log_decay.double().view(-1, *[1] * e.dim()) * e.clamp(min=0).double())
    return torch.where(e >= 0, w, 0.0).float()


class _Chunks:
    """Sequences cut into chunks of C tokens, the last of each padded with zeros."""

    def __init__(self, s, C=CHUNK):
        c, dev = s["case"], s["q"].device
        n, T = c["n"], c["T"]
        self.n, self.C, self.H, self.heads_kv = n, C, c["H"], c["G"]
        cu = torch.arange(n + 1, device=dev) * (T // n) if s["cu"] is None else s["cu"].long()
        lens = cu[1:] - cu[:-1]
        self.lens, counts = lens, (lens + C - 1) // C
        first = counts.cumsum(0) - counts
        total = max(1, sum(-(-x // C) for x in s["lens"]))
        ids = torch.arange(n, device=dev)
        self.seq = torch.repeat_interleave(ids, counts, output_size=total)
        self.at = torch.arange(total, device=dev) - first[self.seq]           # chunk's place in its sequence
        self.i = torch.arange(C, device=dev)
        pos = self.at[:, None] * C + self.i
        self.pos, self.valid = pos, pos < lens[self.seq][:, None]
        self.token = (cu[:-1][self.seq][:, None] + pos).clamp(max=T - 1)
        of = torch.repeat_interleave(ids, lens, output_size=T)
        self.back = first[of] * C + torch.arange(T, device=dev) - cu[:-1][of]
        self.left = torch.where(self.valid, lens[self.seq][:, None] - 1 - pos, -1)  # tokens behind this one
        self.member = (self.seq == ids[:, None]).float()                            # (n, chunks)

    def split(self, t):
        """(tokens, heads, D) -> (H, chunks, C, D) in fp32."""
        t = _rep(t.reshape(-1, t.shape[-2], t.shape[-1]), self.H)
        return torch.where(self.valid[..., None, None], t[self.token].float(), 0.0).permute(2, 0, 1, 3).contiguous()

    def join(self, t, like):
        """(H, chunks, C, D) -> the layout and type of `like`, heads that share one key and value added up."""
        t = t.permute(1, 2, 0, 3).flatten(0, 1)[self.back]
        t = t.unflatten(1, (like.shape[-2], -1)).sum(2) if like.shape[-2] != self.H else t
        return t.reshape(like.shape[:-1] + t.shape[-1:]).to(like.dtype)

    def between(self, log_decay, back=False):
        """decay over the whole chunks between two chunks of one sequence, (H, to, from)."""
        d = self.at[:, None] - self.at
        d = torch.where(self.seq[:, None] == self.seq, -d if back else d, 0) - 1
        return _powers(log_decay, d * self.C)

    def carried(self, log_decay, U, back=False):
        return (self.between(log_decay, back) @ U.flatten(2)).view(U.shape)

    def per_sequence(self, t):
        """(H, chunks, Dk, Dv) summed over each sequence's chunks -> (n, H, Dk, Dv)."""
        return (self.member @ t.transpose(0, 1).flatten(1)).view(self.n, self.H, *t.shape[2:])


def _tr(t):
    return t.transpose(-1, -2)


def _prompt(s):
    ld, scale, c = s["log_decay"], s["scale"], _Chunks(s)
    q, k, v = c.split(s["q"]), c.split(s["k"]), c.split(s["v"])
    h0 = s["pool"][s["slots"].long()] if "slots" in s else None
    low = c.i[:, None] >= c.i
    P = torch.where(low, q @ _tr(k), 0.0) * _powers(ld, c.i[:, None] - c.i)[:, None]
    S = c.carried(ld, _tr(k * _powers(ld, c.C - 1 - c.i)[:, None, :, None]) @ v)
    h = c.per_sequence(_tr(k * _powers(ld, c.left)[..., None]) @ v)
    if h0 is not None:
        S = S + _powers(ld, c.at * c.C)[..., None, None] * h0.transpose(0, 1)[:, c.seq]
        h = h + _powers(ld, c.lens).t()[..., None, None] * h0
    o = scale * (P @ v + _powers(ld, c.i + 1)[:, None, :, None] * (q @ S))
    if "slots" in s:
        s["pool"][s["slots"].long()] = h
    return {"o": c.join(o, s["q"]), "h": s["pool"] if "slots" in s else h}


def _step(s):
    H, rows = s["case"]["H"], s["slots"].long()
    q, k, v = s["q"].float(), _rep(s["k"], H).float(), _rep(s["v"], H).float()
    h = s["pool"][rows] * torch.exp(s["log_decay"])[:, None, None] + k[..., None] * v[..., None, :]
    o = (q[..., None] * h).sum(-2) * s["scale"]
    s["pool"][rows] = h
    return {"o": o.to(s["q"].dtype), "h": s["pool"]}


def _bwd(s):
    ld, c, h0, dh = s["log_decay"], _Chunks(s), s["h0"], s["dh"]
    q, k, v, do = c.split(s["q"]), c.split(s["k"]), c.split(s["v"]), c.split(s["do"]) * s["scale"]
    low, D = c.i[:, None] >= c.i, _powers(ld, c.i[:, None] - c.i)[:, None]
    P, dP = (torch.where(low, a @ _tr(b), 0.0) * D for a, b in ((q, k), (do, v)))
    here, upto = _powers(ld, c.C - 1 - c.i)[:, None, :, None], _powers(ld, c.i + 1)[:, None, :, None]
    S = c.carried(ld, _tr(k * here) @ v) + _powers(ld, c.at * c.C)[..., None, None] * h0.transpose(0, 1)[:, c.seq]
    R = c.carried(ld, _tr(q * upto) @ do, back=True)
    last, tail = dh.transpose(0, 1)[:, c.seq], _powers(ld, c.left)[..., None]  # the final state's gradient, and its way to each token
    dq = dP @ k + upto * (do @ _tr(S))
    dk = _tr(dP) @ q + here * (v @ _tr(R)) + tail * (v @ _tr(last))
    dv = _tr(P) @ do + here * (k @ R) + tail * (k @ last)
    dh0 = c.per_sequence(_tr(q * _powers(ld, c.pos + 1)[..., None]) @ do) + _powers(ld, c.lens).t()[..., None, None] * dh
    return {"dq": c.join(dq, s["q"]), "dk": c.join(dk, s["k"]), "dv": c.join(dv, s["v"]), "dh0": dh0}


def _normed(s):
    r = s["x"].float() + s["residual"].float()
    rstd = (r.square().mean(1) + EPS).rsqrt()
    return r, rstd, r * rstd[:, None] * s["weight"]


def _norm(s):
    r, rstd, y = _normed(s)
    return {"y": y.to(s["x"].dtype), "r": r.to(s["residual"].dtype), "rstd": rstd}


def _groups(y, group):
    rows, D = y.shape
    g = group or D
    return torch.nn.functional.pad(y, (0, -D % g)).view(rows, -1, g)


def _fp8(s):
    r, rstd, y = _normed(s)
    yg = _groups(y, s["case"]["group"])
    scales = yg.abs().amax(2).clamp(min=AMAX_MIN) / FP8_MAX
    q = (yg / scales[..., None]).clamp(-FP8_MAX, FP8_MAX).flatten(1)[:, :y.shape[1]]
    return {"q": q.to(torch.float8_e4m3fn), "scales": scales, "r": r.to(s["residual"].dtype), "rstd": rstd}


def _nbwd(s):
    dy, r, rstd = s["dy"].float(), s["r"].float(), s["rstd"][:, None]
    xh = r * rstd
    g = dy * s["weight"]
    dr = s["dr"].float() + rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    return {"dx": dr.to(s["dy"].dtype), "dr": dr.to(s["r"].dtype), "dw": (dy * xh).sum(0)}


def _clip(s):
    sums = torch.stack([g.float().square().sum() for g in s["grads"]])
    norm = sums.sum().sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    [o.copy_(g.float() * coef) for o, g in zip(s["out"], s["grads"])]
    return {"norm": norm, "clipped": s["flat"]}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op, e = case["op"], _SIZE[case["dtype"]]
    if op in ("step", "prompt", "bwd"):
        H, G, Dk, Dv, n = (case[k] for k in ("H", "G", "Dk", "Dv", "n"))
        T = n if op == "step" else case["T"]
        ins, outs, state = T * (H * Dk + G * (Dk + Dv)) * e, T * H * Dv * e, n * H * Dk * Dv * 4
        if op == "bwd":  # q, k, v, do in, their gradients out (do: its input alone), h0 and dh_out in, dh0 out
            return dict(bytes=2 * ins + outs + 3 * state, flops=12 * T * H * Dk * Dv)
        has = op == "step" or case["packed"]
        return dict(bytes=ins + outs + (2 if has else 1) * state, flops=4 * T * H * Dk * Dv)
    if op == "clip":
        m = sum(math.prod(sh) for sh in _clip_shapes(case))
        return dict(bytes=2 * m * e, flops=3 * m)
    rows, D, r = case["rows"], case["D"], _SIZE[case["res"]]
    m = rows * D
    if op == "nbwd":  # dy, r, dr in; dx and dr out (one tensor where the types are the same)
        return dict(bytes=m * (e + 2 * r + r + (e if e != r else 0)) + 8 * D + 4 * rows, flops=9 * m)
    out = m + 4 * rows * (-(-D // case["group"]) if case["group"] else 1) if op == "fp8" else m * e
    return dict(bytes=m * (e + 2 * r) + out + 4 * D + 4 * rows, flops=(8 if op == "fp8" else 5) * m)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "step":
        return _exact_step(s)
    if op in ("prompt", "bwd"):
        return _exact_tokens(s, op == "bwd")
    if op == "clip":
        total = math.sqrt(sum(float((g.double() ** 2).sum()) for g in s["grads"]))
        f = min(1.0, s["max_norm"] / (total + 1e-6))
        flat, views = _flat(s["grads"], torch.float64)
        for view, g in zip(views, s["grads"]):
            view.copy_(g.double() * f)
        return {"norm": torch.tensor(total, dtype=torch.float64), "clipped": flat}
    w = s["weight"].double()
    if op == "nbwd":
        dy, r = s["dy"].double(), s["r"].double()
        rstd = s["rstd"].double().view(-1, 1)
        dot = torch.einsum("rd,rd,d->r", dy, r, w).view(-1, 1) * rstd / case["D"]
        dr = s["dr"].double() + rstd * dy * w - rstd * rstd * r * dot
        return {"dx": dr, "dr": dr, "dw": torch.einsum("rd,rd,r->d", dy, r, rstd.view(-1))}
    r = torch.add(s["x"].double(), s["residual"].double())
    rstd = 1.0 / torch.sqrt(torch.linalg.vecdot(r, r) / case["D"] + EPS)
    y = torch.einsum("rd,r,d->rd", r, rstd, w)
    if op == "norm":
        return {"y": y, "r": r, "rstd": rstd}
    g = case["group"] or case["D"]
    cols = [y[:, a:a + g] for a in range(0, case["D"], g)]
    scales = torch.stack([b.abs().max(1).values.clamp(min=AMAX_MIN) / FP8_MAX for b in cols], 1)
    q = torch.cat([b / scales[:, i:i + 1] for i, b in enumerate(cols)], 1)
    return {"q": _e4m3(q), "scales": scales, "r": r, "rstd": rstd}


def _e4m3(v):
    """Nearest e4m3 value, ties to even: 3 fraction bits, smallest exponent -6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _exact_step(s):
    H = s["case"]["H"]
    pool, rows = s["pool"].double(), s["slots"].long()
    rep = H // s["k"].shape[1]
    k, v = (s[x].double().repeat_interleave(rep, 1) for x in ("k", "v"))
    h = torch.exp(s["log_decay"].double()).view(H, 1, 1) * pool[rows] + torch.einsum("nhk,nhv->nhkv", k, v)
    pool[rows] = h
    return {"o": torch.einsum("nhk,nhkv->nhv", s["q"].double(), h) * s["scale"], "h": pool}


def _exact_tokens(s, backward):
    """The recurrences token by token, all sequences side by side."""
    c, lens, dev = s["case"], s["lens"], s["q"].device
    H, G, n = c["H"], c["G"], c["n"]
    start = [sum(lens[:i]) for i in range(n)]
    flat = lambda t: t.reshape(c["T"], t.shape[-2], t.shape[-1]).double()  # noqa: E731
    q, k, v = flat(s["q"]), flat(s["k"]).repeat_interleave(H // G, 1), flat(s["v"]).repeat_interleave(H // G, 1)
    lam, scale = torch.exp(s["log_decay"].double()).view(H, 1, 1), s["scale"]
    order = sorted(range(n), key=lambda i: -lens[i])  # longest first: the live ones are a prefix
    at = torch.tensor([start[i] for i in order], device=dev)
    live = [sum(1 for x in lens if x > t) for t in range(max(lens) + 1)]
    pooled = "slots" in s
    rows = s["slots"].long()[order] if pooled else torch.tensor(order, device=dev)
    src = s["pool"] if pooled else s["h0"]
    S = torch.zeros(n, H, c["Dk"], c["Dv"], dtype=torch.float64, device=dev) if src is None else src.double()[rows]
    o = torch.zeros(c["T"], H, c["Dv"], dtype=torch.float64, device=dev)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    do = flat(s["do"]) * scale if backward else None
    for t in range(max(lens)):
        m = live[t]
        i = at[:m] + t
        S[:m] = S[:m] * lam + k[i].unsqueeze(3) * v[i].unsqueeze(2)
        if backward:
            dq[i] = (S[:m] @ do[i].unsqueeze(3)).squeeze(3)
        else:
            o[i] = (q[i].unsqueeze(2) @ S[:m]).squeeze(2) * scale
    shape = lambda t: t.view(*s["q"].shape[:-2], *t.shape[1:])  # noqa: E731
    if not backward:
        if pooled:
            pool = s["pool"].double()
            pool[rows] = S
            return {"o": shape(o), "h": pool}
        h = torch.empty_like(S)
        h[rows] = S
        return {"o": shape(o), "h": h}
    R = s["dh"].double()[rows]
    for t in range(max(lens) - 1, -1, -1):
        m = live[t]
        i = at[:m] + t
        R[:m] += q[i].unsqueeze(3) * do[i].unsqueeze(2)
        dk[i] = (R[:m] @ v[i].unsqueeze(3)).squeeze(3)
        dv[i] = (k[i].unsqueeze(2) @ R[:m]).squeeze(2)
        R[:m] *= lam
    dh0 = torch.empty_like(R)
    dh0[rows] = R
    fold = lambda t: shape(t.unflatten(1, (G, H // G)).sum(2))  # noqa: E731
    return {"dq": shape(dq), "dk": fold(dk), "dv": fold(dv), "dh0": dh0}
