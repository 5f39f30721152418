"""GPU: the global gradient norm and clipping through the C ABI against float64.  Squares are summed
in fp64, so the norm is its fp32 rounding (one u = 2^-24; 2 u are allowed for the square root's
and the sum's own); the factor takes three more roundings and the product one: 6 u, and half a
step, 2^-8, of a bf16 result."""
import math

import pytest
import torch

import layer_forms as lf
import selective_state_space_amd as mb
from gpu_util import require_gpu
from test_gpu_linear_attn import _graph, close, decays

pytestmark = pytest.mark.gpu
U, HB = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def tensors(sizes, dtype, sd=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * sd).to(DT[dtype]) for n in sizes]


def check(got, norm, gs, max_norm, dtype, eps=1e-6):
    total = math.sqrt(sum(float((g.double() ** 2).sum()) for g in gs))
    assert norm.shape == () and abs(float(norm) - total) <= 2 * U * total
    f = min(1.0, max_norm / (total + eps))
    for t, g in zip(got, gs):
        ref = g.double() * f
        close(t, ref, ref.abs() * (6 * U + (HB if dtype == "bf16" else 0)) + 1e-44, "clipped")


SIZES = [[1], [7], [0, 5, 0], [16384], [16385, 3, 1000], list(range(0, 400)), [3] * 250, [200_001, 64, 8, 100_000]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx%d" % (len(s), max(s)))
@pytest.mark.parametrize("max_norm", [0.5, 1e6])
def test_clip(sizes, dtype, max_norm):
    gs = tensors(sizes, dtype)
    c = [g.cuda() for g in gs]
    out, norm = mb.mb_grad_norm_clip(c, max_norm, out=[torch.empty_like(t) for t in c])
    check(out, norm, gs, max_norm, dtype)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(c, gs)), "the gradients were written"
    same, norm2 = mb.mb_grad_norm_clip(c, max_norm)
    assert torch.equal(norm, norm2) and all(a is b for a, b in zip(same, c))
    assert all(torch.equal(a, b) for a, b in zip(c, out)), "in place differs"
    _, norm3 = mb.mb_grad_norm_clip([g.cuda() for g in gs], float("inf"))
    assert torch.equal(norm3, norm)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_clip_views_of_one_buffer(dtype):
    """Odd-sized views into one flat buffer: no start is aligned, neighbours stay untouched."""
    sizes = [5, 300, 17, 40_001, 2]
    gs = tensors(sizes, dtype, seed=3)
    flat = torch.full((sum(sizes) + 2 * len(sizes) + 1,), 9.0, dtype=DT[dtype]).cuda()
    at, views = 1, []
    for g in gs:
        views.append(flat[at:at + g.numel()])
        views[-1].copy_(g)
        at += g.numel() + 2
    _, norm = mb.mb_grad_norm_clip(views, 1.0)
    check(views, norm, gs, 1.0, dtype)
    gaps = flat.clone()
    at = 1
    for g in gs:
        gaps[at:at + g.numel()] = 9.0
        at += g.numel() + 2
    assert bool((gaps == 9.0).all())


def test_clip_far_magnitudes():
    """Squares beyond and below the range of fp32."""
    for sd in (1e30, 1e-30):
        gs = tensors([1000, 70_000], "f32", sd=sd)
        out, norm = mb.mb_grad_norm_clip([g.cuda() for g in gs], sd, eps=0.0)
        check(out, norm, gs, sd, "f32", eps=0.0)


def test_clip_tensor_of_more_than_two_to_the_31_elements():
    big = torch.zeros(2 ** 31 + 12_345, dtype=torch.bfloat16, device="cuda")
    big[-1], big[5] = 3.0, 4.0
    small = torch.zeros(7, dtype=torch.bfloat16, device="cuda")
    out, norm = mb.mb_grad_norm_clip([small, big], 1.0, eps=0.0)
    assert float(norm) == 5.0
    # 3 / 5 and 4 / 5 to half a bf16 step
    assert abs(float(out[1][-1]) - 0.6) <= 0.6 * HB and abs(float(out[1][5]) - 0.8) <= 0.8 * HB
    assert float(out[1].float().abs().max()) <= 0.8 * (1 + HB)


def test_clip_zeros_infinities_and_nan():
    z = [torch.zeros(100).cuda()]
    out, norm = mb.mb_grad_norm_clip(z, 1.0)
    assert float(norm) == 0.0 and bool((out[0] == 0).all())
    a = torch.ones(100).cuda()
    a[3] = float("inf")
    out, norm = mb.mb_grad_norm_clip([a, torch.ones(5).cuda()], 1.0)
    assert float(norm) == math.inf and bool((out[1] == 0).all()) and bool(torch.isnan(out[0][3])) and float(out[0][2]) == 0.0
    a[3] = float("nan")
    out, norm = mb.mb_grad_norm_clip([a, torch.ones(5).cuda()], 1.0)
    assert math.isnan(float(norm)) and bool(torch.isnan(out[1]).all())


def test_clip_without_a_limit_writes_nothing():
    for bad in (float("inf"), float("nan"), 1.0):
        a = torch.arange(100.0).cuda()
        a[3] = bad
        keep = a.clone()
        _, norm = mb.mb_grad_norm_clip([a], float("inf"))
        assert torch.equal(a.nan_to_num(nan=-5.0), keep.nan_to_num(nan=-5.0)) and bool(norm.isfinite()) == (bad == 1.0)
        out, _ = mb.mb_grad_norm_clip([a], float("inf"), out=[torch.zeros_like(a)])
        assert torch.equal(out[0].nan_to_num(nan=-5.0), keep.nan_to_num(nan=-5.0))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off", [(1, 0), (0, 3), (5, 2)], ids=str)
def test_clip_from_one_address_to_another(off, dtype):
    """Gradients and outputs at different distances from a 16-byte address; what lies beside the outputs stays."""
    gs = tensors([40_003, 1, 17, 8], dtype, seed=9)
    src = [torch.zeros(g.numel() + 16, dtype=DT[dtype], device="cuda") for g in gs]
    dst = [torch.full((g.numel() + 16,), 7.0, dtype=DT[dtype], device="cuda") for g in gs]
    a = [t[off[0]:off[0] + g.numel()].copy_(g) for t, g in zip(src, gs)]
    o = [t[off[1]:off[1] + g.numel()] for t, g in zip(dst, gs)]
    out, norm = mb.mb_grad_norm_clip(a, 0.5, out=o)
    check(out, norm, gs, 0.5, dtype)
    for t, g in zip(dst, gs):
        assert bool((t[:off[1]] == 7.0).all()) and bool((t[off[1] + g.numel():] == 7.0).all())


def test_clip_of_tensors_that_share_memory():
    """Gradients that are only read may; a written one may not."""
    flat = torch.randn(5000, generator=torch.Generator().manual_seed(3)).cuda()
    a, b = flat[:4000], flat[2000:]
    out, norm = mb.mb_grad_norm_clip([a, b], 1.0, out=[torch.empty_like(a), torch.empty_like(b)])
    check(out, norm, [a.cpu(), b.cpu()], 1.0, "f32")
    for bad in (lambda: mb.mb_grad_norm_clip([a, b], 1.0), lambda: mb.mb_grad_norm_clip([a, a], 1.0),
                lambda: mb.mb_grad_norm_clip([a, b[2000:]], 1.0, out=[torch.empty_like(a), b[1000:2000]])):
        with pytest.raises(mb.MBError):
            bad()
    mb.mb_grad_norm_clip([a, a[:0], a[:0]], 1.0)


def test_clip_captured_and_replayed():
    c = [g.cuda() for g in tensors([1000, 33, 70_000] + [5] * 200, "bf16")]
    outs = [torch.empty_like(t) for t in c]
    g, (out, norm) = _graph(lambda: mb.mb_grad_norm_clip(c, 1.0, out=outs))
    for r in range(4):
        new = tensors([1000, 33, 70_000] + [5] * 200, "bf16", sd=0.001 + r, seed=r)
        for t, n in zip(c, new):
            t.copy_(n)
        _, want = mb.mb_grad_norm_clip(c, 1.0, out=[torch.empty_like(t) for t in c])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want)
        check(outs, norm, new, 1.0, "bf16")


def test_a_layer_forward_backward_and_clip():
    """The operators as a layer uses them, fp32: norm of the residual stream, projection, linear
    attention, norm, loss; then back through all of it and the clipping, against automatic
    differentiation of the float64 definitions."""
    T, D, H, Dk, lens, eps = 150, 96, 3, 32, [100, 50], 1e-5
    g = torch.Generator().manual_seed(5)
    rn = lambda *s, sd=1.0: (torch.randn(*s, generator=g) * sd).float()
    x, res, w1, W, w2, dy, ld = rn(T, D), rn(T, D), 1 + rn(D, sd=0.2), rn(D, 3 * H * Dk, sd=D ** -0.5), 1 + rn(H * Dk, sd=0.2), rn(T, H * Dk), decays(H)
    cu = torch.tensor([0, 100, 150], dtype=torch.int32).cuda()
    c = {k: t.cuda() for k, t in dict(x=x, res=res, w1=w1, W=W, w2=w2, dy=dy, ld=ld).items()}

    y1, r, rstd1 = mb.mb_rms_norm(c["x"], c["w1"], c["res"], eps=eps)
    qkv = y1 @ c["W"]
    q, k, v = (t.unflatten(1, (H, Dk)) for t in qkv.split(H * Dk, 1))
    o, _ = mb.mb_linear_attn(q, k, v, c["ld"], cu_seqlens=cu)
    of = o.flatten(1)
    y2, _, rstd2 = mb.mb_rms_norm(of, c["w2"], eps=eps)
    do, _, dw2 = mb.mb_rms_norm_bwd(c["dy"], of, rstd2, c["w2"])
    dq, dk, dv, _ = mb.mb_linear_attn_bwd(q, k, v, c["ld"], do.unflatten(1, (H, Dk)), cu_seqlens=cu)
    dqkv = torch.cat([t.flatten(1) for t in (dq, dk, dv)], 1)
    dW = y1.t() @ dqkv
    dx, dr, dw1 = mb.mb_rms_norm_bwd(dqkv @ c["W"].t(), r, rstd1, c["w1"])
    grads, norm = mb.mb_grad_norm_clip([dw1, dW, dw2], 0.1)

    L = {k: t.double().requires_grad_() for k, t in dict(x=x, w1=w1, W=W, w2=w2).items()}
    a, _, _ = lf.rms_norm(L["x"], L["w1"], res.double(), eps)
    q, k, v = (t.unflatten(1, (H, Dk)) for t in (a @ L["W"]).split(H * Dk, 1))
    oo, _ = lf.attn(q, k, v, ld, Dk ** -0.5, lens)
    b, _, _ = lf.rms_norm(oo.flatten(1), L["w2"], None, eps)
    (b * dy.double()).sum().backward()
    want = [L[k].grad for k in ("w1", "W", "w2")]
    total = math.sqrt(sum(float((t ** 2).sum()) for t in want))

    def rel(got, ref):
        return float((got.double().cpu() - ref).norm() / ref.norm())

    # A chain of five fp32 operators, each within a few hundred u of its magnitudes; the norms'
    # rstd amplifies by the rows' size over their mean, about one here: 1e-4 = 1700 u is five
    # times 300 u and leaves no room for a dropped term.
    assert rel(y2, b.detach()) < 1e-4 and rel(dx, L["x"].grad) < 1e-4
    assert abs(float(norm) - total) < 1e-4 * total
    for got, ref in zip(grads, want):
        assert rel(got, ref * (0.1 / total)) < 1e-4
