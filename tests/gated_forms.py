"""Definitions in float64 (torch, CPU) of the gated linear recurrence and of the norm of queries and keys with the
position rotation, each with the bound that fp32 arithmetic keeps to.

Bounds are counted in U = 2^-24, half a step of fp32.
* A gate: e^-v for |v| <= 12 is off by (1.5 |v| + 2) U (the argument's rounding and the exponential's), so s and 1 - s by
  at most 24 U relative to themselves; la = -decay s by 25 U.  a^2 and 1 - a^2 = -e (2 + e), e = e^la - 1, follow
  la: 1 - a^2 is off by 25 U of itself from la and 15 U from its own computation, its root by 20 U, so b by 50 U.
* A state: a step adds |la| a 25 U of the state before (a's own error), 3 U of the sum of magnitudes (the rounding of e,
  of the product and of the sum), and b's error.  Where states of spans are composed, e^S with S a sum of up to 3000 values
  of la is off by 100 U |S| e^S (the sum's rounding: 70 additions one after the other at most), at most 40 U: 60 U of the
  magnitude at any token, not growing from token to token.
* Gradients: the products of these (below, term by term).
"""
import torch

F64 = torch.float64
U = 2.0 ** -24
ROOT_MIN = 2.0 ** -120


def gates(a_gate, x_gate, decay, a_bias, x_bias):
    """(s, 1 - s, la, a, 1 - a^2, beta, i, 1 - i) of every token."""
    va = a_gate if a_bias is None else a_gate + a_bias
    s, not_s = torch.sigmoid(va), torch.sigmoid(-va)
    la = -decay * s
    e = torch.expm1(la)
    less = -e * (2 + e)
    if x_gate is None:
        i, not_i = torch.ones_like(s), torch.zeros_like(s)
    else:
        vx = x_gate if x_bias is None else x_gate + x_bias
        i, not_i = torch.sigmoid(vx), torch.sigmoid(-vx)
    return s, not_s, la, torch.exp(la), less, torch.sqrt(less), i, not_i


def scan(x, a_gate, x_gate, decay, a_bias, x_bias, lens, h0=None):
    """Packed tokens (T, D) in float64.  Returns (y, end states, states before every token, bound of each).  Tokens
    behind sum(lens) give zero rows."""
    _, _, la, a, _, beta, i, _ = gates(a_gate, x_gate, decay, a_bias, x_bias)
    b = beta * i * x
    y, before = torch.zeros_like(x), torch.zeros_like(x)
    ty, tb = torch.zeros_like(x), torch.zeros_like(x)
    ends, tends, t = [], [], 0
    for n_, n in enumerate(lens):
        h = torch.zeros_like(decay) if h0 is None else h0[n_]
        M, E = h.abs(), torch.zeros_like(decay)
        for _ in range(n):
            before[t], tb[t] = h, E + 60 * U * M
            E = a[t] * E + U * (25 * la[t].abs() * a[t] * M + 3 * (a[t] * M + b[t].abs()) + 50 * b[t].abs())
            h, M = a[t] * h + b[t], a[t] * M + b[t].abs()
            y[t], ty[t] = h, E + 60 * U * M
            t += 1
        ends.append(h)
        tends.append(E + (60 * U * M if n else 0 * M))
    z = torch.zeros(0, x.shape[1], dtype=F64)
    return y, torch.stack(ends) if ends else z, before, ty, torch.stack(tends) if tends else z, tb


def scan_bwd(x, a_gate, x_gate, decay, a_bias, x_bias, lens, dy, h0=None, dh=None):
    """Gradients as a dict, and their bounds as another."""
    s, not_s, la, a, less, beta, i, not_i = gates(a_gate, x_gate, decay, a_bias, x_bias)
    b = beta * i * x
    _, _, before, _, _, tb = scan(x, a_gate, x_gate, decay, a_bias, x_bias, lens, h0)
    live = less >= ROOT_MIN
    root = torch.where(live, b / torch.where(live, less, 1.0), 0.0)       # b / beta^2
    G, tG = torch.zeros_like(x), torch.zeros_like(x)
    dh0, th0, t1 = [], [], 0
    for n_, n in enumerate(lens):
        c = torch.zeros_like(decay) if dh is None else dh[n_]
        M, E = c.abs(), torch.zeros_like(decay)
        for t in range(t1 + n - 1, t1 - 1, -1):
            G[t], M = dy[t] + c, dy[t].abs() + M
            E = E + U * 2 * M
            tG[t] = E + 60 * U * M
            c, E, M = a[t] * G[t], a[t] * (E + U * (25 * la[t].abs() + 2) * M), a[t] * M
        dh0.append(c)
        th0.append(E + (60 * U * M if n else 0 * M))
        t1 += n
    tokens = torch.zeros(x.shape[0], 1, dtype=F64)
    tokens[:sum(lens)] = 1
    q = a * before - a * a * root
    dla = G * q * tokens
    # of dla: G's error, that of the state before, and of each term's magnitude 120 U (b, 1 - a^2) and those of a and a^2
    tdla = tG * q.abs() + G.abs() * a * tb + (120 + 60 * la.abs()) * U * G.abs() * (a * before.abs() + a * a * root.abs())
    da, tda = dla * la * not_s, (tdla + 55 * U * dla.abs()) * (la * not_s).abs()
    dx, tdx = G * beta * i * tokens, (tG + 60 * U * G.abs()) * beta * i
    dg, tdg = G * b * not_i * tokens, (tG + 90 * U * G.abs()) * b.abs() * not_i
    terms = (64 + x.shape[0] / 64) * U                   # additions that a sum over tokens passes through
    total = lambda v, tv: (v.sum(0), (tv + terms * v.abs()).sum(0))  # noqa: E731
    out = {"dx": (dx, tdx), "da_gate": (da, tda), "dx_gate": (dg, tdg), "ddecay": total(-dla * s, (tdla + 25 * U * dla.abs()) * s),
           "da_bias": total(da, tda), "dx_bias": total(dg, tdg)}
    z = torch.zeros(0, x.shape[1], dtype=F64)
    out["dh0"] = (torch.stack(dh0) if dh0 else z, torch.stack(th0) if th0 else z)
    return {k: v[0] for k, v in out.items()}, {k: v[1] for k, v in out.items()}


def _pairs(R, inter):
    j = torch.arange(R // 2)
    return (2 * j, 2 * j + 1) if inter else (j, j + R // 2)


def _turn(v, positions, freqs, inter, back):
    """Pairs of v (T, H, D) turned by their positions, and for each element the sum of its pair's magnitudes."""
    R = 2 * freqs.shape[0]
    lo, hi = _pairs(R, inter)
    ang = (positions.to(F64)[:, None] * freqs.to(F64))[:, None] * (-1 if back else 1)
    c, s = torch.cos(ang), torch.sin(ang)
    o, m = v.clone(), v.abs()
    o[..., lo], o[..., hi] = v[..., lo] * c - v[..., hi] * s, v[..., lo] * s + v[..., hi] * c
    m[..., lo] = m[..., hi] = v[..., lo].abs() + v[..., hi].abs()
    return o, m


def norm_rope(x, w, positions, freqs, inter, eps):
    """(T, H, D) in float64.  Returns the result and its bound: a sum of squares passes 16 additions at most one after the
    other in a lane and its tree, so 1 / sqrt(...) is off by 16 U and n by 20 U; an angle, reduced in 64 bits and rounded once, by
    2^-24 pi, its sine and cosine by 6 U more: 40 U of the pair's magnitudes in all."""
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = n if w is None else n * w
    if freqs is None or freqs.numel() == 0:
        return n, 40 * U * n.abs()
    o, m = _turn(n, positions, freqs, inter, False)
    return o, 40 * U * m


def norm_rope_bwd(d, x, w, positions, freqs, inter, eps):
    """(dx, dw) and their bounds."""
    rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xh = x * rstd
    e, me = (d, d.abs()) if freqs is None or freqs.numel() == 0 else _turn(d, positions, freqs, inter, True)
    g = e if w is None else e * w
    mg = me if w is None else me * w.abs()
    dx = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
    # g off by 22 U of its pair, the mean of g xh by 60 U of the mean of magnitudes
    tdx = rstd * (60 * U * mg + 100 * U * xh.abs() * (mg * xh.abs()).mean(-1, keepdim=True))
    rows = x.shape[0] * x.shape[1]
    dw = (e * xh).sum((0, 1))
    tdw = (60 + min(rows, 600) + rows / 64) * U * (me * xh.abs()).sum((0, 1))
    return dx, dw, tdx, tdw
