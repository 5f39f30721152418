"""GPU: the layer operators one behind the other, as a layer uses them: residual norm, projections, norm of queries and keys with the
position rotation, linear attention, and a gated recurrence on its output.  Prompts and single tokens that continue them against the
float64 definitions over whole sequences, and every gradient against float64 differentiation.  Bound: 1e-4 of the largest value of
each result, as for the scans (each operator's own bound is some 1e-5 of its magnitudes; four of them follow each other)."""
import pytest
import torch

import selective_state_space_amd as mb
from gpu_util import assert_close, require_gpu

pytestmark = pytest.mark.gpu
EPS, BASE = 1e-5, 10000.0


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


d_model, H, G, Dk, Dv = 48, 4, 2, 16, 12
D = H * Dv


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s, sd=1.0: torch.randn(*s, generator=g) * sd  # noqa: E731
    w = dict(norm=1 + 0.3 * rn(d_model), qkv=rn(d_model, H * Dk + G * (Dk + Dv), sd=d_model ** -0.5), qn=1 + 0.3 * rn(Dk), kn=1 + 0.3 * rn(Dk),
             mix=rn(D, 3 * D, sd=D ** -0.5), decay=torch.exp(-5 + 6 * torch.rand(D, generator=g)), ab=0.5 * rn(D), xb=0.5 * rn(D))
    w["freqs"] = (BASE ** (-torch.arange(0, Dk, 2, dtype=torch.float64) / Dk)).float()
    w["ld"] = -torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float64) / H).float()
    return w


def defined(x, w, lens, S0, h0):
    """The layer over whole sequences in float64 (differentiable): outputs, attention states, recurrence states."""
    w = {k: v.double() for k, v in w.items()}
    r = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w["norm"]
    q, k, v = (r @ w["qkv"]).split([H * Dk, G * Dk, G * Dv], -1)
    pos = torch.cat([torch.arange(n) for n in lens]).double()
    ang = (pos[:, None] * w["freqs"])[:, None]

    def turned(t, heads, wt):
        t = t.unflatten(-1, (heads, Dk))
        t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS) * wt
        a, b = t[..., :Dk // 2], t[..., Dk // 2:]
        return torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1)

    q, k = turned(q, H, w["qn"]), turned(k, G, w["kn"]).repeat_interleave(H // G, 1)
    v = v.unflatten(-1, (G, Dv)).repeat_interleave(H // G, 1)
    lam = torch.exp(w["ld"]).view(H, 1, 1)
    o, Ss, t = [], [], 0
    for s, n in enumerate(lens):
        S = S0[s]
        for _ in range(n):
            S = lam * S + k[t].unsqueeze(2) * v[t].unsqueeze(1)
            o.append(Dk ** -0.5 * (q[t].unsqueeze(1) @ S).squeeze(1))
            t += 1
        Ss.append(S)
    u, ga, gx = (torch.stack(o).flatten(1) @ w["mix"]).split([D, D, D], -1)
    la = -w["decay"] * torch.sigmoid(ga + w["ab"])
    b = torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(gx + w["xb"]) * u
    ys, hs, t = [], [], 0
    for s, n in enumerate(lens):
        h = h0[s]
        for _ in range(n):
            h = torch.exp(la[t]) * h + b[t]
            ys.append(h)
            t += 1
        hs.append(h)
    return torch.stack(ys), torch.stack(Ss), torch.stack(hs)


def project(x, w):
    y, _, rstd = mb.mb_rms_norm(x, w["norm"], eps=EPS)
    qkv = y @ w["qkv"]
    q, k, v = qkv.split([H * Dk, G * Dk, G * Dv], -1)
    return y, rstd, q.unflatten(-1, (H, Dk)), k.unflatten(-1, (G, Dk)), v.unflatten(-1, (G, Dv))


def test_prompts_and_tokens_that_continue_them():
    """Packed prompts into pool slots, three single tokens for each of them (one sequence pauses for one), then one more prompt on top."""
    lens, more = [70, 1, 260, 129], [3, 3, 2, 3]
    w = weights(1)
    c = {k: v.cuda() for k, v in w.items()}
    n, tail = len(lens), [0, 0, 150, 0]
    total = [a + b + e for a, b, e in zip(lens, more, tail)]
    x = torch.randn(sum(total), d_model, generator=torch.Generator().manual_seed(2))
    first = [sum(total[:i]) for i in range(n)]
    ry, rS, rh = defined(x.double(), w, total, torch.zeros(n, H, Dk, Dv).double(), torch.zeros(n, D).double())
    slots = torch.tensor([4, 0, 5, 2], dtype=torch.int32).cuda()
    S, h = torch.full((6, H, Dk, Dv), 9.0).cuda(), torch.full((6, D), 9.0).cuda()
    got = torch.zeros(sum(total), D)

    def prompts(which, start, count, has):
        rows = torch.cat([torch.arange(first[s] + start[s], first[s] + start[s] + count[s]) for s in which])
        pos = torch.cat([torch.arange(start[s], start[s] + count[s]) for s in which]).int().cuda()
        cu = torch.tensor([sum(count[s] for s in which[:i]) for i in range(len(which) + 1)], dtype=torch.int32).cuda()
        _, _, q, k, v = project(x[rows].cuda(), c)
        q, k = mb.mb_qk_norm_rope(q, k, c["freqs"], pos, q_weight=c["qn"], k_weight=c["kn"], eps=EPS, q_out=q, k_out=k)
        o, _ = mb.mb_linear_attn(q, k, v, c["ld"], cu_seqlens=cu, h0=S, has_h0=has, slots=slots[which])
        u, ga, gx = (o.flatten(1) @ c["mix"]).split([D, D, D], -1)
        y, _ = mb.mb_gated_scan(u, ga, c["decay"], gx, a_bias=c["ab"], x_bias=c["xb"], cu_seqlens=cu, h0=h, has_h0=has, slots=slots[which])
        got[rows] = y.cpu()

    def tokens(which, at):
        rows = torch.tensor([first[s] + at[s] for s in which])
        pos = torch.tensor([at[s] for s in which], dtype=torch.int32).cuda()
        _, _, q, k, v = project(x[rows].cuda(), c)
        q, k = mb.mb_qk_norm_rope(q, k, c["freqs"], pos, q_weight=c["qn"], k_weight=c["kn"], eps=EPS)
        o, _ = mb.mb_linear_attn_step(q, k, v, c["ld"], S, slots=slots[which])
        u, ga, gx = (o.flatten(1) @ c["mix"]).split([D, D, D], -1)
        y, _ = mb.mb_gated_scan_step(u, ga, c["decay"], h, gx, a_bias=c["ab"], x_bias=c["xb"], slots=slots[which])
        got[rows] = y.cpu()

    every = list(range(n))
    prompts(every, [0] * n, lens, torch.zeros(n, dtype=torch.bool).cuda())
    at = list(lens)
    for step in range(3):
        which = [s for s in every if s != 2 or step != 1]
        tokens(which, at)
        for s in which:
            at[s] += 1
    prompts([2], at, tail, None)
    assert_close(got, ry.numpy(), "f32", "outputs")
    assert_close(S[slots.long()], rS.numpy(), "f32", "attention states")
    assert_close(h[slots.long()], rh.numpy(), "f32", "recurrence states")
    for row in (1, 3):
        assert bool((S[row] == 9).all()) and bool((h[row] == 9).all())


def test_gradients_of_the_run():
    lens = [90, 1, 140]
    n, T = len(lens), sum(lens)
    w = weights(3)
    c = {k: v.cuda() for k, v in w.items()}
    g = torch.Generator().manual_seed(4)
    x, dy = torch.randn(T, d_model, generator=g), torch.randn(T, D, generator=g)
    S0, h0 = torch.randn(n, H, Dk, Dv, generator=g), torch.randn(n, D, generator=g)
    leaves = {"x": x, "S0": S0, "h0": h0, **{k: w[k] for k in ("norm", "qkv", "qn", "kn", "mix", "decay", "ab", "xb")}}
    leaves = {k: v.double().requires_grad_() for k, v in leaves.items()}
    y, _, _ = defined(leaves["x"], {**w, **{k: leaves[k] for k in leaves if k in w}}, lens, leaves["S0"], leaves["h0"])
    (y * dy.double()).sum().backward()

    cu = torch.tensor([0, 90, 91, 231], dtype=torch.int32).cuda()
    pos = torch.cat([torch.arange(m) for m in lens]).int().cuda()
    xc, how = x.cuda(), dict(q_weight=c["qn"], k_weight=c["kn"], eps=EPS)
    nrm, rstd, q, k, v = project(xc, c)
    qr, kr = mb.mb_qk_norm_rope(q, k, c["freqs"], pos, **how)
    o, _ = mb.mb_linear_attn(qr, kr, v, c["ld"], cu_seqlens=cu, h0=S0.cuda())
    u, ga, gx = (o.flatten(1) @ c["mix"]).split([D, D, D], -1)
    bias = dict(a_bias=c["ab"], x_bias=c["xb"], cu_seqlens=cu, h0=h0.cuda())
    out, _, kept = mb.mb_gated_scan(u, ga, c["decay"], gx, states=True, **bias)
    assert_close(out, y.detach().numpy(), "f32", "outputs")
    du, dga, dgx, ddecay, dab, dxb, dh0 = mb.mb_gated_scan_bwd(u, ga, c["decay"], dy.cuda(), gx, states=kept, **bias)
    dmixed = torch.cat([du, dga, dgx], -1)
    do = (dmixed @ c["mix"].t()).unflatten(-1, (H, Dv)).contiguous()
    dq, dk, dv, dS0 = mb.mb_linear_attn_bwd(qr, kr, v, c["ld"], do, cu_seqlens=cu, h0=S0.cuda())
    dq, dk, dqn, dkn = mb.mb_qk_norm_rope_bwd(dq, dk, q, k, c["freqs"], pos, **how)
    dqkv = torch.cat([dq.flatten(1), dk.flatten(1), dv.flatten(1)], -1)
    dx, _, dnorm = mb.mb_rms_norm_bwd((dqkv @ c["qkv"].t()).contiguous(), xc, rstd, c["norm"])
    for name, got in dict(x=dx, norm=dnorm, qkv=nrm.t() @ dqkv, qn=dqn, kn=dkn, mix=o.flatten(1).t() @ dmixed, decay=ddecay, ab=dab, xb=dxb, S0=dS0,
                          h0=dh0).items():
        assert_close(got, leaves[name].grad.numpy(), "f32", name)
