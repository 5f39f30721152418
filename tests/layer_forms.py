"""Definitions in float64 (torch, CPU) of the layer operators around the scans, written
token by token and row by row, and the magnitudes their error bounds are counted in."""
import torch

F64 = torch.float64


def attn(q, k, v, log_decay, scale, lens, h0=None):
    """Linear attention on packed tokens (T, heads, width): returns (o, final states).  Tokens
    outside the sequences (behind sum(lens)) give zero rows."""
    H, Dv = q.shape[1], v.shape[2]
    rep = H // k.shape[1]
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    lam = torch.exp(log_decay.to(F64)).view(H, 1, 1)
    o = torch.zeros(q.shape[0], H, Dv, dtype=F64)
    hs, t = [], 0
    for s, n in enumerate(lens):
        S = torch.zeros(H, q.shape[2], Dv, dtype=F64) if h0 is None else h0[s].clone()
        for _ in range(n):
            S = lam * S + k[t].unsqueeze(2) * v[t].unsqueeze(1)
            o[t] = scale * (q[t].unsqueeze(1) @ S).squeeze(1)
            t += 1
        hs.append(S)
    return o, torch.stack(hs) if hs else torch.zeros(0, H, q.shape[2], Dv, dtype=F64)


def attn_bwd(q, k, v, log_decay, scale, lens, do, h0=None, dh=None):
    """Gradients of sum do . o + sum dh . final states: (dq, dk, dv, dh0)."""
    H, G = q.shape[1], k.shape[1]
    rep = H // G
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    lam = torch.exp(log_decay.to(F64)).view(H, 1, 1)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    out, t0 = [], 0
    for s, n in enumerate(lens):
        zero = torch.zeros(H, q.shape[2], v.shape[2], dtype=F64)
        S = zero if h0 is None else h0[s].clone()
        for t in range(t0, t0 + n):
            S = lam * S + k[t].unsqueeze(2) * v[t].unsqueeze(1)
            dq[t] = scale * (S @ do[t].unsqueeze(2)).squeeze(2)
        R = zero if dh is None else dh[s].clone()
        for t in range(t0 + n - 1, t0 - 1, -1):
            R = R + scale * q[t].unsqueeze(2) * do[t].unsqueeze(1)
            dk[t] = (R @ v[t].unsqueeze(2)).squeeze(2)
            dv[t] = (k[t].unsqueeze(1) @ R).squeeze(1)
            R = lam * R
        out.append(R)
        t0 += n
    fold = lambda x: x.unflatten(1, (G, rep)).sum(2)
    return dq, fold(dk), fold(dv), torch.stack(out)


def rms_norm(x, weight, residual, eps):
    r = x if residual is None else x + residual
    rstd = 1.0 / torch.sqrt((r * r).mean(-1) + eps)
    y = r * rstd.unsqueeze(-1)
    return (y if weight is None else y * weight), r, rstd


def rms_norm_bwd(dy, r, rstd, weight, dr_in):
    xh = r * rstd.unsqueeze(-1)
    g = dy if weight is None else dy * weight
    dr = rstd.unsqueeze(-1) * (g - xh * (g * xh).mean(-1, keepdim=True))
    return (dr if dr_in is None else dr + dr_in), (dy * xh).reshape(-1, dy.shape[-1]).sum(0)
