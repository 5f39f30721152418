"""GPU: the layer operators at the ends of the sizes that they take.  Bounds as in
tests/test_gpu_linear_attn.py and tests/test_gpu_rms_norm.py."""
import pytest
import torch

import layer_forms as lf
import selective_state_space_amd as mb
from gpu_util import require_gpu
from test_gpu_linear_attn import bound, close

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_one_sequence_of_almost_two_to_the_31_tokens():
    """Length and number of segments together pass 2^31.  With a decay of e^-0.25 a token, what lies 300 tokens away weighs
    e^-75 and is left out of the windows' references, which are compared in their middle thirds."""
    T, ld = 2 ** 31 - 5, torch.tensor([-0.25])
    g = torch.Generator(device="cuda").manual_seed(1)

    def fill():
        return torch.empty(1, T, 1, 1, dtype=torch.bfloat16, device="cuda").uniform_(-2.0, 2.0, generator=g)

    q, k, v, do = fill(), fill(), fill(), fill()
    o = torch.full_like(q, float("nan"))
    _, h = mb.mb_linear_attn(q, k, v, ld.cuda(), scale=0.5, o=o)
    grads = mb.mb_linear_attn_bwd(q, k, v, ld.cuda(), do, scale=0.5, dq=torch.full_like(q, float("nan")))
    for t in (o, grads[0]):
        assert not any(bool(torch.isnan(p).any()) for p in t.view(-1).split(2 ** 28)), "tokens that were not written"
    # the first tokens, some of the segments' borders (2^20 tokens each), the last tokens
    for at in (300, 2 ** 20, 2 ** 20 * 777, 2 ** 30, 2 ** 20 * 2047, T - 300):
        w = slice(at - 300, at + 300)
        d = [t[0, w].cpu().double() for t in (q, k, v, do)]
        a = [t.abs() for t in d]
        first, last = 0 if at == 300 else 300, 600 if at == T - 300 else 300      # tokens with all that reaches them
        ro, rh = lf.attn(*d[:3], ld, 0.5, [600])
        Mo, Mh = lf.attn(*a[:3], ld, 0.5, [600])
        tol = bound("bf16", 1, [600], Mo, ro)
        close(o[0, w][first:], ro[first:], tol[first:], "o at %d" % at)
        if at == T - 300:
            close(h, rh, bound("f32", 1, [600], Mh, rh), "h")
        ref, mag = lf.attn_bwd(*d[:3], ld, 0.5, [600], d[3]), lf.attn_bwd(*a[:3], ld, 0.5, [600], a[3])
        for name, got, r, M, part in zip(("dq", "dk", "dv"), grads, ref, mag, (slice(first, 600), slice(0, last), slice(0, last))):
            close(got[0, w][part], r[part], bound("bf16", 5, [600], M, r)[part], name + " at %d" % at)


def _pairs(n, G, D, H, dtype, seed, share=1.0):
    """Inputs of n packed sequences of zero, one or two tokens; `share` of them may have some."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = torch.randint(0, 3, (n,), generator=g, device="cuda")
    lens *= torch.rand(n, generator=g, device="cuda") < share
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    cu[1:] = lens.cumsum(0)
    T = int(cu[-1])
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)
    return lens, cu, T, rn(T, H, D), rn(T, G, D), rn(T, G, D), rn(T, H, D)


def _pairs_forward(q, k, v, ld, scale, lens, cu):
    """o and the end states of sequences of at most two tokens."""
    lam = torch.exp(ld.double().cuda()).view(-1, 1)
    first = cu[:-1][lens > 0].long()
    second = cu[:-1][lens > 1].long() + 1
    h = torch.zeros(lens.numel(), q.shape[1], q.shape[2], v.shape[2], dtype=F64, device="cuda")
    h[lens > 0] = k[first].unsqueeze(3) * v[first].unsqueeze(2)
    o = torch.zeros(q.shape[0], q.shape[1], v.shape[2], dtype=F64, device="cuda").index_add(
        0, first, scale * (q[first] * k[first]).sum(2, keepdim=True) * v[first])
    o = o.index_add(0, second, scale * (q[second] * k[second]).sum(2, keepdim=True) * v[second])
    o = o.index_add(0, second, scale * lam * (q[second] * k[second - 1]).sum(2, keepdim=True) * v[second - 1])
    h[lens > 1] = h[lens > 1] * lam.unsqueeze(2) + k[second].unsqueeze(3) * v[second].unsqueeze(2)
    return o, h


def _check_pairs(n, H, D, seed, share=1.0):
    """Forward and backward of n such sequences; returns their tokens."""
    scale = 0.5
    ld = -torch.arange(1.0, H + 1) / H
    lens, cu, T, q, k, v, do = _pairs(n, H, D, H, torch.float32, seed, share)
    o, h = mb.mb_linear_attn(q, k, v, ld.cuda(), scale=scale, cu_seqlens=cu)
    grads = mb.mb_linear_attn_bwd(q, k, v, ld.cuda(), do, scale=scale, cu_seqlens=cu)
    # magnitudes are added up over at most two tokens of four products each: 16 roundings are more than there are, and
    # the decay's exponent is off by less than 2 u of one
    tol = lambda M: 20 * 2.0 ** -24 * M
    L = [t.double() for t in (q, k, v)]
    A = [t.abs() for t in L]
    for got, r, M, name in zip((o, h), _pairs_forward(*L, ld, scale, lens, cu), _pairs_forward(*A, ld, scale, lens, cu), "oh"):
        assert bool(((got - r).abs() <= tol(M)).all()), name
    del o, h, got, r, M
    auto, mag = [], []
    for src, d, out in ((L, do.double(), auto), (A, do.double().abs(), mag)):
        leaves = [t.requires_grad_() for t in src]
        (_pairs_forward(*leaves, ld, scale, lens, cu)[0] * d).sum().backward()
        out += [t.grad for t in leaves]
    for got, r, M, name in zip(grads, auto, mag, ("dq", "dk", "dv")):
        assert bool(((got - r).abs() <= tol(M)).all()), name
    assert not bool(grads[3].isnan().any())
    return T


def test_more_workgroups_than_a_launch_takes():
    """2^20 sequences of 8 heads: as many threads as a grid may not have, forward and backward."""
    assert _check_pairs(2 ** 20, 8, 4, 2) > 2 ** 19


def test_many_sequences_of_few_tokens():
    """Hundreds of thousands of sequences, nearly all empty: a workgroup finds its own without looking through the
    others'.  And so many heads that no sequence is cut, whose segments come from the table."""
    assert _check_pairs(300_000, 8, 4, 5, share=0.003) <= 1024
    assert 1024 < _check_pairs(20_000, 512, 2, 6, share=0.1) < 4000


def test_offsets_of_few_tokens_out_of_range_stay_inside():
    """Offsets outside [0, T] where no sequence is cut count as the nearest bound, decreasing ones touch nothing outside."""
    T, H, D = 900, 2, 16
    g = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn(T, H, D, generator=g) for _ in range(3))
    ld = torch.tensor([-0.1, -1.0])
    cu = torch.tensor([-7, 300, 300, 2000, 3000], dtype=torch.int32).cuda()       # [0, 300), empty, [300, 900), empty
    o, h = mb.mb_linear_attn(q.cuda(), k.cuda(), v.cuda(), ld.cuda(), cu_seqlens=cu)
    a = [t.double() for t in (q, k, v)]
    ro, rh = lf.attn(*a, ld, D ** -0.5, [300, 0, 600, 0])
    Mo, Mh = lf.attn(*[t.abs() for t in a], ld, D ** -0.5, [300, 0, 600, 0])
    close(o, ro, bound("f32", D, [600], Mo, ro), "o")
    close(h, rh, bound("f32", D, [600], Mh, rh), "h")
    room = torch.full((T + 256, H, D), 7.0, device="cuda")
    cu = torch.tensor([900, 0, 900, 100, 2 ** 31 - 1, -2 ** 31, 5], dtype=torch.int64).to(torch.int32).cuda()
    mb.mb_linear_attn(q.cuda(), k.cuda(), v.cuda(), ld.cuda(), cu_seqlens=cu, o=room[128:-128])
    assert bool((room[:128] == 7.0).all()) and bool((room[-128:] == 7.0).all())


def test_more_workgroups_than_a_launch_takes_step():
    """2^20 rows of 16 heads, states in reversed slots of a pool."""
    n, H, D, scale = 2 ** 20, 16, 4, 0.5
    ld = -torch.arange(1.0, H + 1) / H
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(n, H, D, generator=g, device="cuda") for _ in range(3))
    pool = torch.randn(n, H, D, D, generator=g, device="cuda")
    slots = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")
    start = pool.flip(0)
    o, h = mb.mb_linear_attn_step(q, k, v, ld.cuda(), pool, scale=scale, slots=slots)
    assert h is pool
    lam = torch.exp(ld.double().cuda()).view(-1, 1, 1)
    U = 2.0 ** -24
    for part in torch.arange(n, device="cuda").chunk(4):
        Q, K, V, S = (t[part].double() for t in (q, k, v, start))
        S0, S = S.abs() * lam + (K.unsqueeze(3) * V.unsqueeze(2)).abs(), S * lam + K.unsqueeze(3) * V.unsqueeze(2)
        assert bool(((pool.flip(0)[part] - S).abs() <= 16 * U * S0).all()), "h"
        want, M = scale * (Q.unsqueeze(2) @ S).squeeze(2), scale * (Q.abs().unsqueeze(2) @ S0).squeeze(2)
        assert bool(((o[part] - want).abs() <= (D + 64) * U * M).all()), "o"


@pytest.mark.parametrize("rows,D", [(2 ** 26 + 5, 2), (2 ** 26 + 5, 8), (2 ** 22 + 3, 8200)], ids=str)
def test_more_rows_than_a_launch_takes(rows, D):
    """A row in a wave (four to a workgroup) and in 1024 threads: rows on both sides of the border of two launches."""
    u = 2.0 ** -24
    x = torch.ones(rows, D, dtype=torch.bfloat16, device="cuda")
    border = 2 ** 26 - 4 if D <= 8 else 2 ** 22 - 1
    some = torch.cat([torch.arange(8), torch.arange(border - 8, border + 6), torch.arange(rows - 8, rows)])
    some = some[some < rows].unique().cuda()
    x[some] = torch.randn(some.numel(), D, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    r = x[some].double()
    rs = (r.square().mean(1) + 1e-5).rsqrt()
    if D <= 8:
        y, _, rstd = mb.mb_rms_norm(x)
        assert bool(((y[some] - r * rs[:, None]).abs() <= (2.0 ** -8 + 64 * u) * (r * rs[:, None]).abs()).all())
        one = float((1 / torch.tensor(1 + 1e-5).double().sqrt()).bfloat16())
        assert int((y != one).any(1).sum()) <= some.numel(), "rows that were not written"
        del y
    q, s, _, rstd = mb.mb_rms_norm_fp8(x, group=32)
    assert bool(((rstd[some] - rs).abs() <= 40 * u * rs).all())
    per = s[some].double().repeat_interleave(32, 1)[:, :D]
    want = r * rs[:, None]
    assert bool(((q[some].double() * per - want).abs() <= (2.0 ** -4 + 140 * u) * want.abs() + per * 2.0 ** -10).all())
    # every other row is ones: its code is 448 everywhere
    other = torch.cat([(part.view(torch.uint8) == 0x7e).all(1) for part in q.split(2 ** 18 if D > 8 else 2 ** 24)])
    other[some] = True
    assert bool(other.all()), "rows that were not written"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 7, 600, 1500, 2048, 2049, 9000])
def test_norm_of_rows_whose_squares_leave_the_range(D, dtype):
    """Finite rows of 1e18 to the largest values and, without an eps that covers them, down to subnormal ones; single large
    values among ordinary ones; ordinary rows beside them; zeros and a row with an infinity as ever."""
    u, hb = 2.0 ** -24, 2.0 ** -8 if dtype == "bf16" else 0.0
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    sizes = [1.0, 1e18, 1e19, 1e20, 1e30, 8e37, 1e-18, 1e-20, 1e-25, 1e-37, 2.0 ** -135]
    g = torch.Generator().manual_seed(9)
    x = (torch.randn(len(sizes) + 2, D, generator=g).clamp(-3.0, 3.0).sign() * (0.5 + torch.rand(len(sizes) + 2, D, generator=g)))
    x[:len(sizes)] *= torch.tensor(sizes)[:, None]
    x[-2, D // 2] = 3e38
    x[-1, D // 2] = -2e19
    x, w = x.to(dt), 1 + 0.3 * torch.randn(D, generator=g)
    for eps in (1e-5, 1e-33, 1e-41, 0.0, 1e30):
        e = float(torch.tensor(eps))                          # what the kernel takes
        r = x.double()
        rs = 1 / torch.sqrt(r.square().mean(1) + e)
        ry = r * rs[:, None] * w.double()
        # the last size is zero in bf16: with an eps of 0 the formula itself is zero times infinity there
        some = torch.isfinite(ry).all(1)
        assert int(some.sum()) >= len(sizes) + (1 if dtype == "bf16" and eps == 0.0 else 2)
        r, rs, ry = r[some], rs[some], ry[some]
        for group in (None, 0, 32):
            if group is None:
                y, _, rstd = mb.mb_rms_norm(x.cuda(), w.cuda(), eps=eps)
                assert bool(torch.isnan(y[~some]).all())
                y = y[some]
                # a product below the normal range is rounded to 2^-150
                close(y, ry, (64 * u + hb) * ry.abs() + 2.0 ** (-134 if dtype == "bf16" else -148), "y, eps %g" % eps)
            else:
                q, s, _, rstd = mb.mb_rms_norm_fp8(x.cuda(), w.cuda(), group=group, eps=eps)
                assert bool(torch.isnan(q[~some].float()).all()) and bool(torch.isnan(s[~some]).all())
                q, s, n = q.cpu()[some], s[some], group or D
                yg = torch.nn.functional.pad(ry, (0, -D % n)).view(ry.shape[0], -1, n)
                sc = yg.abs().amax(2).clamp(min=2.0 ** -96) / 448
                close(s, sc, 70 * u * sc, "scales, eps %g" % eps)
                per = sc.repeat_interleave(n, 1)[:, :D]
                close(q.cpu().double() * s.cpu().double().repeat_interleave(n, 1)[:, :D], ry,
                      ry.abs() * (2.0 ** -4 + 140 * u) + per * 2.0 ** -10, "q, eps %g" % eps)
            got = rstd.double().cpu()[some]
            ok = rs < 3.4e38                                  # beyond: infinite in fp32
            close(got[ok], rs[ok], 40 * u * rs[ok] + 2.0 ** -149, "rstd, eps %g" % eps)
            assert bool((got[~ok] > 3.4e38).all())
    # with the forward's rstd the gradient is that of the rows' directions
    r32 = x.float().cuda()
    y, _, rstd = mb.mb_rms_norm(r32[:6].contiguous(), w.cuda(), eps=1e-5)
    dy = torch.randn(6, D, generator=g)
    dx, _, dw = mb.mb_rms_norm_bwd(dy.cuda(), r32[:6].contiguous(), rstd, w.cuda())
    rr, rw = lf.rms_norm_bwd(dy.double(), x[:6].double(), rstd.double().cpu(), w.double(), None)
    xh, gw = x[:6].double() * rstd.double().cpu()[:, None], dy.double() * w.double()
    mag = rstd.double().cpu()[:, None] * (gw.abs() + xh.abs() * (gw * xh).abs().mean(1, keepdim=True))
    close(dx, rr, 100 * u * mag + 2.0 ** -148, "dx")
    close(dw, rw, 106 * u * (dy.double() * xh).abs().sum(0) + 1e-30, "dw")


def test_norm_of_zeros_and_infinities_is_the_formulas():
    x = torch.zeros(3, 40)
    x[1, 3], x[2, 5] = float("inf"), float("nan")
    x[1, 4] = 3e38
    y, _, rstd = mb.mb_rms_norm(x.cuda(), eps=1e-5)
    assert bool((y[0] == 0).all()) and float(rstd[0]) == pytest.approx(1e5 ** 0.5, rel=1e-6)
    assert float(rstd[1]) == 0.0 and bool(torch.isnan(y[1, 3])) and bool((y[1, 4:] == 0).all())
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(rstd[2]))
    y, _, rstd = mb.mb_rms_norm(x[:1].cuda(), eps=0.0)
    assert bool(torch.isinf(rstd).all()) and bool(torch.isnan(y).all())
