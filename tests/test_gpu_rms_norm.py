"""GPU: the residual RMS norm, its 8-bit output and its backward through the C ABI against the
float64 definitions of tests/layer_forms.py.

Bounds in u = 2^-24 (half a step of fp32): a sum of D squares (all positive) passes at most 64
additions in a thread and its tree, so rstd is within 40 u and y within 64 u of its value; a bf16
output adds half a step, 2^-8, an e4m3 one 2^-4 of a normal value or 2^-10 of the scale.  dr adds
up three terms whose fp32 errors are within 100 u of their magnitudes; dw sums the rows' products
one after the other: (100 + rows) u of the sum of magnitudes."""
import pytest
import torch

import layer_forms as lf
import selective_state_space_amd as mb
from gpu_util import require_gpu
from test_gpu_linear_attn import _graph, close

pytestmark = pytest.mark.gpu
U, HB = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def make(seed, rows, D, dtype, res, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s, d=torch.float32: (torch.randn(*s, generator=g) * scale).to(d)
    return rn(rows, D, d=DT[dtype]), rn(rows, D, d=DT[res]), 1 + 0.3 * torch.randn(D, generator=g)


TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]
SHAPES = [(1, 1), (3, 7), (4, 768), (5, 512), (7, 513), (66, 1001), (9, 1100), (5, 1840), (3, 2048), (2, 2049), (5, 4104), (2, 8192), (3, 8200), (2, 16384)]


def rounded(v, dtype, u=1):
    return v.abs() * (u * U + (HB if dtype == "bf16" else 0.0))


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm(types, shape):
    (dtype, res), (rows, D) = types, shape
    x, r0, w = make(1, rows, D, dtype, res)
    for weight, residual in ((w, r0), (None, r0), (w, None)):
        y, r, rstd = mb.mb_rms_norm(x.cuda(), None if weight is None else weight.cuda(), None if residual is None else residual.cuda(), eps=EPS)
        ry, rr, rs = lf.rms_norm(x.double(), None if weight is None else weight.double(), None if residual is None else residual.double(), EPS)
        # the addition's own rounding moves r by u of itself, whatever cancelled
        close(y, ry, rounded(ry, dtype, 64) + 1e-30, "y")
        close(rstd, rs, 40 * U * rs, "rstd")
        close(r, rr, rounded(rr, res if residual is not None else dtype, 1) + 1e-30, "r")


@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_norm_strided_unaligned_and_in_place(types):
    dtype, res = types
    rows, D = 9, 200
    x, r0, w = make(2, rows, D, dtype, res)
    want = mb.mb_rms_norm(x.cuda(), w.cuda(), r0.cuda(), eps=EPS)
    for lead, width in ((0, 264), (1, 203), (3, 208)):
        wide = torch.full((rows, width + lead), float("nan"), dtype=DT[dtype]).cuda()
        view = wide[:, lead:lead + D]
        view.copy_(x)
        r = r0.clone().cuda()
        y, r2, rstd = mb.mb_rms_norm(view, w.cuda(), r, eps=EPS, residual_out=r)
        assert r2 is r and torch.equal(r, want[1])
        # vector and element kernels add the squares up in another order
        close(y, want[0].double().cpu(), rounded(want[0].double().cpu(), dtype, 64) * 2 + 1e-30, "y")
        assert bool(torch.isnan(wide).sum() == rows * (width + lead - D))


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 1), (5, 100), (6, 768), (4, 1001), (5, 1840), (3, 2048), (3, 2056), (2, 8192), (2, 9000)], ids=str)
def test_norm_8_bits(types, group, shape):
    (dtype, res), (rows, D) = types, shape
    x, r0, w = make(3, rows, D, dtype, res)
    x[:, : D // 3] *= 1e-3                       # groups of unlike sizes, and subnormal codes per row
    r0[:, : D // 3] *= 1e-3
    q, s, r, rstd = mb.mb_rms_norm_fp8(x.cuda(), w.cuda(), r0.cuda(), group=group, eps=EPS)
    ry, rr, rs = lf.rms_norm(x.double(), w.double(), r0.double(), EPS)
    g = group or D
    yg = torch.nn.functional.pad(ry, (0, -D % g)).view(rows, -1, g)
    sc = yg.abs().amax(2).clamp(min=2.0 ** -96) / 448
    assert q.dtype == torch.float8_e4m3fn and s.shape == sc.shape
    close(s, sc, 70 * U * sc, "scales")
    per = sc.repeat_interleave(g, 1)[:, :D]
    close(q.cpu().double() * s.cpu().double().repeat_interleave(g, 1)[:, :D], ry,
          ry.abs() * (2.0 ** -4 + 140 * U) + per * 2.0 ** -10, "q")
    close(r, rr, rounded(rr, res, 1) + 1e-30, "r")
    close(rstd, rs, 40 * U * rs, "rstd")
    # what the codes say is the nearest e4m3 value of the quotient, but where the fp32 error crosses a border
    v = ry / per
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    near = (torch.round(v / step) * step).clamp(-448, 448)
    border = ((v / step - torch.floor(v / step)) - 0.5).abs() * step <= 200 * U * v.abs() + 1e-12
    assert bool(((q.cpu().double() == near) | border).all())


@pytest.mark.parametrize("group", [0, 32])
def test_norm_8_bits_of_zeros_infinities_and_nan(group):
    x = torch.zeros(4, 64)
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3] = torch.arange(64.0)
    for width in (64, 65):                       # vector and element kernels
        buf = torch.zeros(4, width).cuda()
        view = buf[:, :64]
        view.copy_(x)
        q, s, r, rstd = mb.mb_rms_norm_fp8(view, group=group)
        q = q.cpu().double()
        assert bool((q[0] == 0).all()) and bool((s[0].cpu() == 2.0 ** -96 / 448).all())
        assert bool(torch.isnan(q[1]).all()) and bool(torch.isnan(s[1]).all())
        # an infinite element: rstd 0, itself NaN, the others zero; its group's scale NaN
        assert bool(torch.isnan(s[2, 0])) and bool(torch.isnan(q[2, :32]).all())
        assert bool(torch.isfinite(q[3]).all()) and float(q[3].max()) == 448.0


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("shape", SHAPES + [(2500, 40), (1030, 2056)], ids=str)
def test_norm_backward(types, shape):
    (dtype, res), (rows, D) = types, shape
    dy, r, w = make(4, rows, D, dtype, res)
    dr_in = make(5, rows, D, dtype, res)[1]
    rstd = (r.double().square().mean(1) + EPS).rsqrt().float()
    for weight, inn in ((w, dr_in), (None, None)):
        c = lambda t: None if t is None else t.cuda()
        dx, dr, dw = mb.mb_rms_norm_bwd(dy.cuda(), r.cuda(), rstd.cuda(), c(weight), c(inn))
        D64 = lambda t: None if t is None else t.double()
        rr, rw = lf.rms_norm_bwd(dy.double(), r.double(), rstd.double(), D64(weight), D64(inn))
        g = dy.double() * (1.0 if weight is None else weight.double())
        xh = r.double() * rstd.double()[:, None]
        mag = rstd.double()[:, None] * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) + (0 if inn is None else inn.double().abs())
        close(dr, rr, 100 * U * mag + (HB if res == "bf16" else 0) * rr.abs() + 1e-30, "dr")
        close(dx, rr, 100 * U * mag + (HB if dtype == "bf16" else 0) * rr.abs() + 1e-30, "dx")
        close(dw, rw, (100 + rows) * U * (dy.double() * xh).abs().sum(0) + 1e-30, "dw")
        again = mb.mb_rms_norm_bwd(dy.cuda(), r.cuda(), rstd.cuda(), c(weight), c(inn))
        assert torch.equal(again[2], dw) and torch.equal(again[1], dr)
    stream = dr_in.clone().cuda()                # the stream's gradient updated in place
    dx, dr, dw = mb.mb_rms_norm_bwd(dy.cuda(), r.cuda(), rstd.cuda(), w.cuda(), stream, dr=stream)
    assert dr is stream
    want = mb.mb_rms_norm_bwd(dy.cuda(), r.cuda(), rstd.cuda(), w.cuda(), dr_in.cuda())
    assert torch.equal(dr, want[1]) and torch.equal(dw, want[2])


def test_norm_no_rows():
    for D in (8, 20):
        x, w = torch.empty(0, D).cuda(), torch.ones(D).cuda()
        y, r, rstd = mb.mb_rms_norm(x, w, x)
        assert y.shape == (0, D) and rstd.shape == (0,)
        assert mb.mb_rms_norm_fp8(x, w, group=32)[1].shape == (0, 1)
        dx, dr, dw = mb.mb_rms_norm_bwd(x, x, rstd, w)
        assert bool((dw == 0).all())


def test_norm_captured_and_replayed():
    x, r0, w = (t.cuda() for t in make(6, 600, 768, "bf16", "f32"))
    dy = torch.randn(600, 768).bfloat16().cuda()

    def fn():
        y, r, rstd = mb.mb_rms_norm(x, w, r0)
        q, s, _, _ = mb.mb_rms_norm_fp8(x, w, r0, group=64)
        return (y, r, rstd, q.view(torch.uint8), s) + mb.mb_rms_norm_bwd(dy, r, rstd, w, r)

    g, out = _graph(fn)
    for k in range(4):
        a, b, _ = make(10 + k, 600, 768, "bf16", "f32")
        x.copy_(a)
        r0.copy_(b)
        want = fn()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), "replay %d" % k


def test_norm_rows_behind_two_to_the_31_elements():
    D, rows = 4096, 2 ** 19 + 3
    x = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 2 ** 31
    last = torch.randn(3, D).bfloat16()
    x[-3:] = last.cuda()
    y, r, rstd = mb.mb_rms_norm(x, eps=EPS)
    ry, _, rs = lf.rms_norm(last.double(), None, None, EPS)
    assert r is x
    close(y[-3:], ry, rounded(ry, "bf16", 64), "y")
    close(rstd[-3:], rs, 40 * U * rs, "rstd")
    del y
    q, s, _, _ = mb.mb_rms_norm_fp8(x, group=128, eps=EPS)
    close(q[-3:].cpu().double() * s[-3:].cpu().double().repeat_interleave(128, 1), ry,
          ry.abs() * (2.0 ** -4 + 140 * U) + s[-3:].cpu().double().repeat_interleave(128, 1) * 2.0 ** -10, "q")
