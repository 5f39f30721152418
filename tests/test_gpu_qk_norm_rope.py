"""GPU: the norm of queries and keys with the position rotation, and its backward, through the C ABI against the float64
definitions and bounds of tests/gated_forms.py; a bf16 output adds half a step, 2^-8 of its value."""
import pytest
import torch

import gated_forms as gf
import selective_state_space_amd as mb
from gpu_util import require_gpu
from test_gpu_linear_attn import _graph, close

pytestmark = pytest.mark.gpu
HB = 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
TINY = 1e-37


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def make(seed, T, Hq, Hk, D, R, dtype, far=5000):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = DT[dtype]
    d = dict(q=rn(T, Hq, D).to(t), k=rn(T, max(Hk, 1), D).to(t), dq=rn(T, Hq, D).to(t), dk=rn(T, max(Hk, 1), D).to(t), wq=1 + 0.3 * rn(D), wk=1 + 0.3 * rn(D))
    d["freqs"] = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))).float()
    d["pos"] = torch.randint(-far, far, (T,), generator=g, dtype=torch.int32)
    return d


def tol(bound, ref, dtype):
    return bound + (HB if dtype == "bf16" else 0.0) * ref.abs() + TINY


def check(d, out, name, dtype, inter, eps=EPS, w=True, pos=None, R=True):
    x = d[name].double()
    r, t = gf.norm_rope(x, d["w" + name].double() if w else None, d["pos"] if pos is None else pos, d["freqs"] if R else None, inter, eps)
    close(out.reshape(x.shape), r, tol(t, r, dtype), name)


# T, query heads, key heads, width, rotated columns
SHAPES = [(1, 1, 1, 1, 0), (1, 16, 4, 128, 128), (3, 2, 1, 2, 2), (5, 4, 2, 64, 64), (70, 6, 2, 80, 32), (9, 3, 3, 33, 10), (257, 1, 1, 16, 8),
          (4, 8, 8, 256, 256), (3, 2, 1, 512, 128), (2, 1, 0, 511, 510), (33, 5, 1, 100, 100), (6, 2, 2, 96, 48), (130, 12, 3, 40, 40), (2, 300, 7, 24, 24),
          (5, 3, 1, 72, 0), (4, 2, 2, 128, 16), (7, 1, 1, 192, 96), (1000, 4, 1, 128, 64)]


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype, inter):
    T, Hq, Hk, D, R = shape
    d = make(1, *shape, dtype)
    c = {k: v.cuda() for k, v in d.items()}
    k = c["k"] if Hk else None
    q_, k_ = mb.mb_qk_norm_rope(c["q"], k, c["freqs"], c["pos"], q_weight=c["wq"], k_weight=c["wk"] if Hk else None, interleaved=inter, eps=EPS)
    check(d, q_, "q", dtype, inter)
    if Hk:
        check(d, k_, "k", dtype, inter)
    else:
        assert k_ is None
    # no weights, no positions: places; no rotation
    q_, _ = mb.mb_qk_norm_rope(c["q"], k, c["freqs"], interleaved=inter, eps=EPS)
    check(d, q_, "q", dtype, inter, w=False, pos=torch.arange(T))
    q_, _ = mb.mb_qk_norm_rope(c["q"], k, q_weight=c["wq"], eps=EPS)
    check(d, q_, "q", dtype, inter, R=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 1, 4, 8])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 32), (36, 12), (128, 128)])
def test_views_and_in_place(D, R, off, dtype):
    """Columns of a projection from any element, batches with places counted from zero, in place; the values are left alone."""
    B, L, Hq, Hk = 2, 37, 4, 2
    d = make(2, B * L, Hq, Hk, D, R, dtype)
    width = (Hq + 2 * Hk) * D + off + 3
    buf = torch.full((B, L, width), 5.0, dtype=DT[dtype])
    buf[..., off:off + Hq * D] = d["q"].view(B, L, -1)
    buf[..., off + Hq * D:off + (Hq + Hk) * D] = d["k"].view(B, L, -1)
    buf = buf.cuda()
    q, k = buf[..., off:off + Hq * D].unflatten(-1, (Hq, D)), buf[..., off + Hq * D:off + (Hq + Hk) * D].unflatten(-1, (Hk, D))
    kw = dict(q_weight=d["wq"].cuda(), k_weight=d["wk"].cuda(), eps=EPS)
    pos = torch.arange(L).repeat(B)
    q1, k1 = mb.mb_qk_norm_rope(q, k, d["freqs"].cuda(), **kw)
    check(d, q1, "q", dtype, False, pos=pos)
    check(d, k1, "k", dtype, False, pos=pos)
    dqk = [d[n].view(B, L, *d[n].shape[1:]).cuda() for n in ("dq", "dk")]
    back = mb.mb_qk_norm_rope_bwd(*dqk, q, k, d["freqs"].cuda(), **kw)
    for name, got, gw in (("q", back[0], back[2]), ("k", back[1], back[3])):
        r, rw, t, tw = gf.norm_rope_bwd(d["d" + name].double(), d[name].double(), d["w" + name].double(), pos, d["freqs"], False, EPS)
        close(got.reshape(r.shape), r, tol(t, r, dtype), "d" + name)
        close(gw, rw, tol(tw, rw, "f32"), "dw" + name)
    keep = buf.clone()
    q2, k2 = mb.mb_qk_norm_rope(q, k, d["freqs"].cuda(), q_out=q, k_out=k, **kw)
    assert q2 is q and k2 is k and torch.equal(q2, q1) and torch.equal(k2, k1)
    assert torch.equal(buf[..., :off], keep[..., :off]) and torch.equal(buf[..., off + (Hq + Hk) * D:], keep[..., off + (Hq + Hk) * D:])


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES + [(3000, 2, 1, 64, 64)], ids=str)
def test_backward(shape, dtype, inter):
    T, Hq, Hk, D, R = shape
    d = make(3, *shape, dtype)
    c = {k: v.cuda() for k, v in d.items()}
    keys = (c["dk"], c["k"], c["wk"]) if Hk else (None, None, None)
    for weights in (True, False):
        kw = dict(interleaved=inter, eps=EPS, **(dict(q_weight=c["wq"], k_weight=keys[2]) if weights else {}))
        out = mb.mb_qk_norm_rope_bwd(c["dq"], keys[0], c["q"], keys[1], c["freqs"], c["pos"], **kw)
        for name, got, gw in (("q", out[0], out[2]), ("k", out[1], out[3])):
            if name == "k" and not Hk:
                assert got is None and gw is None
                continue
            w = d["w" + name].double() if weights else None
            r, rw, t, tw = gf.norm_rope_bwd(d["d" + name].double(), d[name].double(), w, d["pos"], d["freqs"], inter, EPS)
            close(got, r, tol(t, r, dtype), "d" + name)
            if weights:
                close(gw, rw, tol(tw, rw, "f32"), "dw" + name)
            else:
                assert gw is None
        again = mb.mb_qk_norm_rope_bwd(c["dq"], keys[0], c["q"], keys[1], c["freqs"], c["pos"], **kw)
        assert all(a is b or torch.equal(a, b) for a, b in zip(out, again)), "two runs differ"


def test_gradients_against_differences():
    T, H, D, R = 5, 2, 12, 8
    d = make(4, T, H, H, D, R, "f32")
    out = mb.mb_qk_norm_rope_bwd(d["dq"].cuda(), d["dk"].cuda(), d["q"].cuda(), d["k"].cuda(), d["freqs"].cuda(), d["pos"].cuda(),
                                 q_weight=d["wq"].cuda(), k_weight=d["wk"].cuda(), eps=EPS)
    g = torch.Generator().manual_seed(1)
    for name, gx, gw in (("q", out[0], out[2]), ("k", out[1], out[3])):
        x, w, up = d[name].double(), d["w" + name].double(), d["d" + name].double()
        loss = lambda x, w: float((up * gf.norm_rope(x, w, d["pos"], d["freqs"], False, EPS)[0]).sum())  # noqa: E731
        dx, dw = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(w.shape, generator=g, dtype=torch.float64)
        e = 1e-5
        for num, got, way in (((loss(x + e * dx, w) - loss(x - e * dx, w)) / (2 * e), gx, dx), ((loss(x, w + e * dw) - loss(x, w - e * dw)) / (2 * e), gw, dw)):
            prod = got.double().cpu() * way
            assert abs(num - float(prod.sum())) <= 2e-5 * float(prod.abs().sum()) + 1e-7


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("D", [64, 34])
def test_far_positions_keep_their_angle(D, inter):
    """Up to the ends of the integers: the angle's turns are reduced in 64 bits."""
    pos = torch.tensor([0, 1, -1, 10 ** 6, 10 ** 6 + 1, -10 ** 8, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    d = make(5, len(pos), 3, 1, D, D, "f32")
    d["pos"] = pos
    c = {k: v.cuda() for k, v in d.items()}
    q_, k_ = mb.mb_qk_norm_rope(c["q"], c["k"], c["freqs"], c["pos"], q_weight=c["wq"], k_weight=c["wk"], interleaved=inter, eps=EPS)
    # position * freq in 64 bits is off by 2^-53 of at most 2^31, and so is the definition's own: 2^-22 each, 8 U together
    for name, out in (("q", q_), ("k", k_)):
        r, t = gf.norm_rope(d[name].double(), d["w" + name].double(), pos, d["freqs"], inter, EPS)
        close(out, r, 1.3 * t + TINY, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 50])
def test_large_small_zero_infinite_and_nan_heads(D, dtype):
    """Squares outside fp32's range, zeros, and what is not finite stays in its own head."""
    T, H, R = 6, 3, 16
    d = make(6, T, H, 1, D, R, dtype)
    scale = torch.ones(T, H, 1)
    scale[0, 0], scale[1, 1], scale[2, 2], scale[3, 0] = 1e30, 1e-30, 0.0, 3e37
    d["q"] = (d["q"].float() * scale).to(DT[dtype])
    c = {k: v.cuda() for k, v in d.items()}
    for eps in (EPS, 0.0, 1e-30):
        q_, _ = mb.mb_qk_norm_rope(c["q"], None, c["freqs"], c["pos"], q_weight=c["wq"], eps=eps)
        x = d["q"].double()
        if eps == 0.0:
            x[2, 2] = 1.0                                   # zeros with no eps: 0 / 0
            q_[2, 2] = gf.norm_rope(x, d["wq"].double(), d["pos"], d["freqs"], False, eps)[0][2, 2].to(q_)
        r, t = gf.norm_rope(x, d["wq"].double(), d["pos"], d["freqs"], False, eps)
        close(q_, r, tol(t, r, dtype) + 2 * gf.U * r.abs(), "q")
    back = mb.mb_qk_norm_rope_bwd(c["dq"], None, c["q"], None, c["freqs"], c["pos"], q_weight=c["wq"], eps=EPS)
    r, rw, t, tw = gf.norm_rope_bwd(d["dq"].double(), d["q"].double(), d["wq"].double(), d["pos"], d["freqs"], False, EPS)
    close(back[0], r, tol(t, r, dtype), "dq")
    close(back[2], rw, tol(tw, rw, "f32"), "dwq")
    good, _ = mb.mb_qk_norm_rope(c["q"], None, c["freqs"], c["pos"], q_weight=c["wq"], eps=EPS)
    for bad in (float("nan"), float("inf")):
        e = c["q"].clone()
        e[4, 1, 7] = bad
        q_, _ = mb.mb_qk_norm_rope(e, None, c["freqs"], c["pos"], q_weight=c["wq"], eps=EPS)
        assert bool(torch.isnan(q_[4, 1]).any())
        q_[4, 1] = good[4, 1]
        assert torch.equal(q_, good)


def test_no_tokens():
    q, k = torch.empty(0, 4, 16).cuda(), torch.empty(0, 2, 16).cuda()
    f, w = torch.ones(4).cuda(), torch.ones(16).cuda()
    a, b = mb.mb_qk_norm_rope(q, k, f)
    assert a.shape == q.shape and b.shape == k.shape
    out = mb.mb_qk_norm_rope_bwd(q, k, q, k, f, q_weight=w, k_weight=w)
    assert bool((out[2] == 0).all()) and bool((out[3] == 0).all())


def test_graph_replays():
    d = make(7, 300, 8, 2, 64, 64, "bf16")
    c = {k: v.cuda() for k, v in d.items()}
    kw = dict(q_weight=c["wq"], k_weight=c["wk"], eps=EPS)

    def both():
        return mb.mb_qk_norm_rope(c["q"], c["k"], c["freqs"], c["pos"], **kw) + \
            mb.mb_qk_norm_rope_bwd(c["dq"], c["dk"], c["q"], c["k"], c["freqs"], c["pos"], **kw)

    want = [t.clone() for t in both()]
    graph, out = _graph(both)
    for i in range(4):
        for t in out:
            t.fill_(float("nan"))
        both()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_rows_past_32_bit_offsets():
    T, Hq, D, stride = 1100, 2, 64, (1 << 22) - 8
    buf = torch.zeros(T * stride, dtype=torch.bfloat16, device="cuda")              # 9 GB
    d = make(8, T, Hq, 1, D, D, "bf16")
    q = buf.view(T, stride)[:, :Hq * D].unflatten(1, (Hq, D))
    q.copy_(d["q"])
    mb.mb_qk_norm_rope(q, None, d["freqs"].cuda(), d["pos"].cuda(), q_weight=d["wq"].cuda(), eps=EPS, q_out=q)
    check(d, q.contiguous(), "q", "bf16", False)


def test_more_tokens_than_a_launch_takes():
    """2^28 tokens and some: more threads than one grid has; in place, one head of one pair."""
    T, D, n = (1 << 28) + 37, 2, 300
    q = torch.ones(T, 1, D, dtype=torch.bfloat16, device="cuda")                   # 1 GB
    f = torch.full((1,), 0.37).cuda()
    places = torch.cat([torch.arange(n), torch.arange(T - n, T)])
    q[places.cuda()] = torch.randn(2 * n, 1, D, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    want, _ = mb.mb_qk_norm_rope(q[places.cuda()], None, f, places.int().cuda(), eps=EPS)
    mb.mb_qk_norm_rope(q, None, f, eps=EPS, q_out=q)
    assert torch.equal(q[places.cuda()], want)
    rest = q[n:T - n:1021, 0].float()
    # (1, 1) turned: two squares that add up to 2 / (1 + EPS), each value off by half a step, (1 + HB)^2 of its square
    assert bool((((rest * rest).sum(1) - 2.0).abs() <= 2 * (2 * HB + HB * HB) + 3 * EPS).all())
