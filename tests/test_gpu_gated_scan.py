"""GPU: the gated linear recurrence, its single-token step and its backward through the C ABI against the float64
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
TINY = 1e-37            # results and bounds that leave fp32's range


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def make(seed, T, D, dtype, n, gate=True, bias=True, decay="mixed"):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s, d=torch.float32: torch.randn(*s, generator=g).to(d)  # noqa: E731
    t = DT[dtype]
    d = dict(x=rn(T, D, d=t), a_gate=(2 * rn(T, D)).to(t), x_gate=rn(T, D, d=t), dy=rn(T, D, d=t), h0=rn(n, D), dh=rn(n, D),
             a_bias=0.5 * rn(D), x_bias=0.5 * rn(D))
    lo, hi = {"mixed": (-7.0, 2.0), "slow": (-12.0, -9.0), "fast": (1.0, 4.0)}[decay]
    d["decay"] = torch.exp(lo + (hi - lo) * torch.rand(D, generator=g))
    if not gate:
        d["x_gate"] = d["x_bias"] = None
    if not bias:
        d["a_bias"] = d["x_bias"] = None
    return d


def wide(d):
    return [None if d[k] is None else d[k].double() for k in ("x", "a_gate", "x_gate", "decay", "a_bias", "x_bias")]


def dev(t, *lead):
    return None if t is None else (t.view(*lead, *t.shape[1:]) if lead else t).cuda()


def offsets(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)


def tol(bound, ref, dtype):
    return bound + (HB if dtype == "bf16" else 0.0) * ref.abs() + TINY


# (batch, L) or packed lengths, D: lengths from nothing to several tiles and groups of tiles, on and beside their borders
SPECS = [((1, 1), 1), ((1, 1), 64), ((3, 5), 7), ((1, 64), 64), ((2, 63), 66), ((1, 65), 130), ((1, 127), 40), ((2, 128), 65), ((1, 129), 33),
         ((2, 300), 100), ((1, 2000), 70), ((1, 2200), 16), ((2, 2304), 8), ((1, 6000), 3), ((4, 1024), 64),
         ([5, 0, 1, 64, 200], 64), ([0, 0], 5), ([130, 0, 0, 126, 1, 255], 96), ([1] * 300, 20), ([2500, 3, 0, 2100], 34), ([128, 128, 0, 256], 128),
         ([0, 700, 0], 129), ([7] * 40 + [0] * 90 + [400], 10)]


def ident(c):
    s, D = c
    return ("+".join(map(str, s)) if len(s) < 8 else "%d seqs" % len(s)) + ("p" if isinstance(s, list) else "") + "x%d" % D


def unpack(spec):
    packed = isinstance(spec, list)
    return packed, (spec if packed else [spec[1]] * spec[0]), (() if packed else spec)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", SPECS, ids=ident)
def test_forward(case, dtype):
    (spec, D), (packed, lens, lead) = case, unpack(case[0])
    T, n = sum(lens), len(lens)
    for gate, bias, decay, h0 in ((True, True, "mixed", True), (False, True, "slow", False), (True, False, "fast", True)):
        d = make(1, T, D, dtype, n, gate, bias and gate, decay)
        cu = offsets(lens).cuda() if packed else None
        y, h, st = mb.mb_gated_scan(dev(d["x"], *lead), dev(d["a_gate"], *lead), d["decay"].cuda(), dev(d["x_gate"], *lead), a_bias=dev(d["a_bias"]),
                                    x_bias=dev(d["x_bias"]), cu_seqlens=cu, h0=d["h0"].cuda() if h0 else None, states=True)
        ry, rh, rb, ty, th, tb = gf.scan(*wide(d), lens, d["h0"].double() if h0 else None)
        close(y.reshape(T, D), ry, tol(ty, ry, dtype), "y")
        close(h, rh, tol(th, rh, "f32"), "h")
        assert st.shape == (-(-T // 64), D)
        close(st, rb[::64], tol(tb[::64], rb[::64], "f32"), "states")
        again = mb.mb_gated_scan(dev(d["x"], *lead), dev(d["a_gate"], *lead), d["decay"].cuda(), dev(d["x_gate"], *lead), a_bias=dev(d["a_bias"]),
                                 x_bias=dev(d["x_bias"]), cu_seqlens=cu, h0=d["h0"].cuda() if h0 else None)
        assert torch.equal(again[0], y) and torch.equal(again[1], h), "two runs differ, or by the states"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off,D", [(0, 64), (2, 64), (1, 50), (0, 33), (3, 96)])
def test_views_pools_and_rows_outside(off, D, dtype):
    """Columns of one projection, from any element, packed sequences whose states lie in a pool, and tokens in front of
    the first and behind the last sequence, which hold NaN."""
    lens, head, tail = [40, 0, 1, 300, 129], 3, 70
    n, T = len(lens), sum([40, 0, 1, 300, 129])
    d = make(5, T, D, dtype, n)
    buf = torch.full((head + T + tail, 3 * D + off + 5), float("nan"), dtype=DT[dtype])
    for i, k in enumerate(("x", "a_gate", "x_gate")):
        buf[head:head + T, off + i * D:off + (i + 1) * D] = d[k]
    x, a, g = buf.cuda()[:, off:off + 3 * D].split([D, D, D], 1)
    slots, has = torch.tensor([6, 0, 3, -1, 9], dtype=torch.int32), torch.tensor([1, 0, 1, 1, 1], dtype=torch.uint8)
    pool = torch.randn(8, D, generator=torch.Generator().manual_seed(3))
    start = torch.stack([pool[s] if 0 <= s < 8 and f else torch.zeros(D) for s, f in zip(slots.tolist(), has.tolist())])
    got, y = pool.clone().cuda(), torch.full((head + T + tail, D), 7.0, dtype=DT[dtype]).cuda()
    cu = (offsets(lens) + head).int().cuda()
    bias = dict(a_bias=d["a_bias"].cuda(), x_bias=d["x_bias"].cuda())
    y2, h2 = mb.mb_gated_scan(x, a, d["decay"].cuda(), g, cu_seqlens=cu, h0=got, has_h0=has.cuda(), slots=slots.cuda(), y=y, **bias)
    assert y2 is y and h2 is got
    assert bool((y[:head] == 7.0).all()) and bool((y[head + T:] == 7.0).all()), "rows outside the sequences were written"
    ry, rh, _, ty, th, _ = gf.scan(*wide(d), lens, start.double())
    close(y[head:head + T], ry, tol(ty, ry, dtype), "y")
    for s, slot in enumerate(slots.tolist()):
        if 0 <= slot < 8:
            close(got[slot], rh[s], tol(th[s], rh[s], "f32"), "slot %d" % slot)
    for slot in (1, 2, 4, 5, 7):
        assert torch.equal(got[slot].cpu(), pool[slot]), "an unnamed slot was written"
    # the backward of the same rows: zeros outside
    dy = torch.full((head + T + tail, D), float("nan"), dtype=DT[dtype])
    dy[head:head + T] = d["dy"]
    out = mb.mb_gated_scan_bwd(x, a, d["decay"].cuda(), dy.cuda(), g, cu_seqlens=cu, h0=start.cuda(), dh_out=d["dh"].cuda(), **bias)
    ref, bound = gf.scan_bwd(*wide(d), lens, d["dy"].double(), start.double(), d["dh"].double())
    for name, got_ in zip(("dx", "da_gate", "dx_gate", "ddecay", "da_bias", "dx_bias", "dh0"), out):
        if name in ("dx", "da_gate", "dx_gate"):
            assert bool((got_[:head] == 0).all()) and bool((got_[head + T:] == 0).all()), name
            got_ = got_[head:head + T]
        close(got_, ref[name], tol(bound[name], ref[name], dtype if got_.dtype == DT[dtype] else "f32"), name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_split_chains_and_steps(dtype):
    """A sequence in two prompts and single tokens, the state handed on in place, equals one call to its bounds."""
    L, a, b, D = 300, 173, 290, 72
    d = make(11, L, D, dtype, 1)
    c = {k: d[k].cuda() for k in ("x", "a_gate", "x_gate", "decay", "a_bias", "x_bias")}
    bias = dict(a_bias=c["a_bias"], x_bias=c["x_bias"])
    h, ys = d["h0"].clone().cuda(), []
    for i, j in ((0, a), (a, b)):
        y, h2 = mb.mb_gated_scan(*(c[k][None, i:j] for k in ("x", "a_gate")), c["decay"], c["x_gate"][None, i:j], h0=h, h_out=h, **bias)
        assert h2 is h
        ys.append(y[0])
    for t in range(b, L):
        y, _ = mb.mb_gated_scan_step(c["x"][t:t + 1], c["a_gate"][t:t + 1], c["decay"], h, c["x_gate"][t:t + 1], **bias)
        ys.append(y)
    ry, rh, _, ty, th, _ = gf.scan(*wide(d), [L], d["h0"].double())
    close(torch.cat(ys), ry, tol(ty, ry, dtype), "y")
    close(h, rh, tol(th, rh, "f32"), "h")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,D,off", [(1, 1, 0), (1, 1536, 0), (5, 33, 1), (70, 64, 2), (3, 130, 3), (300, 20, 0), (2, 8, 1)])
def test_step(n, D, off, dtype):
    d = make(7, n, D, dtype, n)
    buf = torch.full((n, 3 * D + off), float("nan"), dtype=DT[dtype])
    for i, k in enumerate(("x", "a_gate", "x_gate")):
        buf[:, off + i * D:off + (i + 1) * D] = d[k]
    x, a, g = buf.cuda()[:, off:].split([D, D, D], 1)
    bias = dict(a_bias=d["a_bias"].cuda(), x_bias=d["x_bias"].cuda())
    ry, rh, _, ty, th, _ = gf.scan(*wide(d), [1] * n, d["h0"].double())
    h = d["h0"].cuda()
    out = torch.full_like(h, 5.0)
    y, h2 = mb.mb_gated_scan_step(x, a, d["decay"].cuda(), h, g, h_out=out, **bias)
    assert h2 is out and torch.equal(h.cpu(), d["h0"])
    close(y, ry, tol(ty, ry, dtype), "y")
    close(out, rh, tol(th, rh, "f32"), "h")
    y2, h3 = mb.mb_gated_scan_step(x, a, d["decay"].cuda(), h, g, **bias)
    assert h3 is h and torch.equal(h, out) and torch.equal(y, y2)
    # a pool: scattered rows, one sequence without a row
    slots = torch.randperm(n + 4, generator=torch.Generator().manual_seed(2))[:n].int()
    slots[-1] = -1 if n > 1 else slots[-1]
    pool = torch.randn(n + 4, D, generator=torch.Generator().manual_seed(4))
    start = torch.stack([pool[s] if s >= 0 else torch.zeros(D) for s in slots.tolist()])
    got = pool.clone().cuda()
    y, _ = mb.mb_gated_scan_step(x, a, d["decay"].cuda(), got, g, slots=slots.cuda(), **bias)
    ry, rh, _, ty, th, _ = gf.scan(*wide(d), [1] * n, start.double())
    close(y, ry, tol(ty, ry, dtype), "y")
    named = set(slots.tolist())
    for s, slot in enumerate(slots.tolist()):
        if slot >= 0:
            close(got[slot], rh[s], tol(th[s], rh[s], "f32"), "slot")
    for slot in set(range(n + 4)) - named:
        assert torch.equal(got[slot].cpu(), pool[slot])
    # no input gate, no biases
    d = make(8, n, D, dtype, n, gate=False, bias=False)
    y, h = mb.mb_gated_scan_step(d["x"].cuda(), d["a_gate"].cuda(), d["decay"].cuda(), d["h0"].cuda())
    ry, rh, _, ty, th, _ = gf.scan(*wide(d), [1] * n, d["h0"].double())
    close(y, ry, tol(ty, ry, dtype), "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", SPECS, ids=ident)
def test_backward(case, dtype):
    (spec, D), (packed, lens, lead) = case, unpack(case[0])
    T, n = sum(lens), len(lens)
    for gate, bias, decay, has in ((True, True, "mixed", True), (False, False, "slow", False), (True, False, "fast", True)):
        d = make(21, T, D, dtype, n, gate, bias, decay)
        cu = offsets(lens).cuda() if packed else None
        ins = [dev(d["x"], *lead), dev(d["a_gate"], *lead), d["decay"].cuda()]
        g, dy = dev(d["x_gate"], *lead), dev(d["dy"], *lead)
        kw = dict(a_bias=dev(d["a_bias"]), x_bias=dev(d["x_bias"]), cu_seqlens=cu, h0=d["h0"].cuda() if has else None)
        h0, dh = (d["h0"].double(), d["dh"].double()) if has else (None, None)
        ref, bound = gf.scan_bwd(*wide(d), lens, d["dy"].double(), h0, dh)
        kept = mb.mb_gated_scan(*ins, g, states=True, **kw)[2]
        runs = []
        for states in (kept, None, kept):
            out = mb.mb_gated_scan_bwd(*ins, dy, g, dh_out=d["dh"].cuda() if has else None, states=states, **kw)
            runs.append(out)
            for name, got in zip(("dx", "da_gate", "dx_gate", "ddecay", "da_bias", "dx_bias", "dh0"), out):
                if name == "dx_gate" and not gate or name.endswith("bias") and not (bias and (gate or name[1] == "a")):
                    assert got is None
                    continue
                close(got.reshape(ref[name].shape), ref[name], tol(bound[name], ref[name], dtype if name in ("dx", "da_gate", "dx_gate") else "f32"), name)
        assert all(a is b or torch.equal(a, b) for a, b in zip(runs[0], runs[2])), "two runs differ"


def test_gradients_against_differences():
    """Every gradient but dx_bias' like against central differences of the GPU forward's 64-bit definition."""
    lens, D = [37, 0, 70], 4
    T, n = sum(lens), len(lens)
    d = make(31, T, D, "f32", n)
    out = mb.mb_gated_scan_bwd(d["x"].cuda(), d["a_gate"].cuda(), d["decay"].cuda(), d["dy"].cuda(), d["x_gate"].cuda(), a_bias=d["a_bias"].cuda(),
                               x_bias=d["x_bias"].cuda(), cu_seqlens=offsets(lens).cuda(), h0=d["h0"].cuda(), dh_out=d["dh"].cuda())
    names = ("x", "a_gate", "x_gate", "decay", "a_bias", "x_bias", "h0")
    base = {k: d[k].double() for k in names}

    def loss(v):
        y, h = gf.scan(v["x"], v["a_gate"], v["x_gate"], v["decay"], v["a_bias"], v["x_bias"], lens, v["h0"])[:2]
        return float((d["dy"].double() * y).sum() + (d["dh"].double() * h).sum())

    g = torch.Generator().manual_seed(1)
    for name, got in zip(names, (out[0], out[1], out[2], out[3], out[4], out[5], out[6])):
        way = torch.randn(base[name].shape, generator=g, dtype=torch.float64)
        if name == "decay":
            way = way * base[name]
        eps = 1e-5
        num = (loss({**base, name: base[name] + eps * way}) - loss({**base, name: base[name] - eps * way})) / (2 * eps)
        ana = float((got.double().cpu() * way).sum())
        # differences in 64 bits are off by eps^2 of a third derivative and 1e-16 / eps: 1e-8 of the magnitudes added up, and the
        # gradient itself by some 1e-5 of them
        mag = float((got.double().cpu() * way).abs().sum())
        assert abs(num - ana) <= 3e-5 * mag + 1e-7, (name, num, ana)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinities_and_nan_stay_where_they_are(dtype):
    """One in a token reaches its channel from that token to the end of its sequence, and nothing else; in the backward
    those in front of it too, by the state they lead to, but no other sequence or channel."""
    lens, D = [200, 300, 150], 70
    T, n = sum(lens), len(lens)
    d = make(41, T, D, dtype, n)
    t, c = 333, 5
    cu = offsets(lens).cuda()
    for bad in (float("nan"), float("inf")):
        for key in ("x", "a_gate", "x_gate"):
            if bad == float("inf") and key != "x":
                continue                                  # an open gate, no infinity
            e = {k: v.clone() for k, v in d.items()}
            e[key][t, c] = bad
            kw = dict(a_bias=e["a_bias"].cuda(), x_bias=e["x_bias"].cuda(), cu_seqlens=cu, h0=e["h0"].cuda())
            y, h = mb.mb_gated_scan(e["x"].cuda(), e["a_gate"].cuda(), e["decay"].cuda(), e["x_gate"].cuda(), **kw)
            ry, rh = (v.cpu() for v in mb.mb_gated_scan(d["x"].cuda(), d["a_gate"].cuda(), d["decay"].cuda(), d["x_gate"].cuda(), **kw))
            y, h = y.cpu(), h.cpu()
            assert not bool(torch.isfinite(y[t:500, c]).any()) and not bool(torch.isfinite(h[1, c]))
            y[t:500, c], h[1, c] = ry[t:500, c], rh[1, c]
            assert torch.equal(y, ry) and torch.equal(h, rh)
            args = lambda v: (v["x"].cuda(), v["a_gate"].cuda(), v["decay"].cuda(), v["dy"].cuda(), v["x_gate"].cuda())  # noqa: E731
            out = mb.mb_gated_scan_bwd(*args(e), dh_out=e["dh"].cuda(), **kw)
            want = mb.mb_gated_scan_bwd(*args(d), dh_out=e["dh"].cuda(), **kw)
            for name, got, ref in zip(("dx", "da_gate", "dx_gate", "ddecay", "da_bias", "dx_bias", "dh0"), out, want):
                got, ref = got.cpu().clone(), ref.cpu()
                if name in ("dx", "da_gate", "dx_gate"):
                    got[200:500, c] = ref[200:500, c]
                elif name == "dh0":
                    got[1, c] = ref[1, c]
                else:
                    assert not bool(torch.isfinite(got[c])) or name == "dx_bias" and key == "a_gate" or bad == float("inf"), name
                    got[c] = ref[c]
                assert torch.equal(got, ref), (name, key, bad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_closed_open_and_extreme_gates(dtype):
    """Gates far outside where they move, no decay at all, infinite decay: finite, and as the limits say."""
    T, D = 140, 8
    d = make(51, T, D, dtype, 1)
    d["decay"] = torch.tensor([0.0, float("inf"), 1e-30, 100.0, 1.0, 1.0, 1.0, 1.0])
    d["a_gate"][:, 4], d["a_gate"][:, 5], d["x_gate"][:, 6], d["x_gate"][:, 7] = -200.0, 200.0, -200.0, 200.0
    c = {k: d[k].cuda() for k in ("x", "a_gate", "x_gate", "decay")}
    y, h = mb.mb_gated_scan(c["x"][None], c["a_gate"][None], c["decay"], c["x_gate"][None], h0=d["h0"].cuda())
    y, h0 = y[0].cpu().double(), d["h0"][0].double()
    assert bool(torch.isfinite(y).all())
    half = HB if dtype == "bf16" else 2.0 ** -23
    si = torch.sigmoid(d["x_gate"].double())
    assert bool(((y[:, 0] - h0[0]).abs() <= half * h0[0].abs()).all())                     # no decay: the state stays
    assert bool(((y[:, 1] - si[:, 1] * d["x"][:, 1].double()).abs() <= (2 * half + 24 * gf.U) * y[:, 1].abs() + TINY).all())   # no memory
    assert bool(((y[:, 2] - h0[2]).abs() <= half * h0[2].abs() + 1e-12).all())
    assert bool(((y[:, 4] - h0[4]).abs() <= half * h0[4].abs() + 1e-12).all())             # closed: no decay, no input
    assert bool(((y[:, 6] - h0[6] * torch.exp(-torch.cumsum(torch.sigmoid(d["a_gate"][:, 6].double()), 0))).abs() <= 2 * half * y[:, 6].abs() + 1e-5).all())
    out = mb.mb_gated_scan_bwd(c["x"][None], c["a_gate"][None], c["decay"], d["dy"].cuda()[None], c["x_gate"][None], h0=d["h0"].cuda(),
                               dh_out=d["dh"].cuda())
    for name, got in zip(("dx", "da_gate", "dx_gate", "ddecay"), out):
        got = got.cpu().double().reshape(-1, D)
        keep = [0, 2, 3, 4, 5, 6, 7]                    # infinite decay has no derivative by it
        assert bool(torch.isfinite(got[:, keep]).all()), name
    assert bool((out[1].cpu()[0, :, 0] == 0).all()) and bool((out[0].cpu()[0, :, 0] == 0).all())
    # with no decay ddecay is that of the state alone: beta, which is zero, is left out
    G = torch.flip(torch.cumsum(torch.flip(d["dy"][:, 0].double(), (0,)), 0), (0,)) + d["dh"][0, 0].double()
    want = -(G * h0[0] * torch.sigmoid(d["a_gate"][:, 0].double())).sum()
    assert abs(float(out[3][0]) - float(want)) <= 1e-4 * float((G * h0[0]).abs().sum())


def test_offsets_out_of_range_stay_inside():
    """Offsets outside [0, T] count as the nearest bound; decreasing ones touch nothing outside."""
    T, D = 700, 32
    d = make(12, T, D, "f32", 4)
    c = [d[k].cuda() for k in ("x", "a_gate", "decay", "x_gate")]
    kw = dict(a_bias=d["a_bias"].cuda(), x_bias=d["x_bias"].cuda(), h0=d["h0"].cuda())
    y, h = mb.mb_gated_scan(*c, cu_seqlens=torch.tensor([-5, 300, 300, 1500, 2000], dtype=torch.int32).cuda(), **kw)
    ry, rh, _, ty, th, _ = gf.scan(*wide(d), [300, 0, 400, 0], d["h0"].double())
    close(y, ry, tol(ty, ry, "f32"), "y")
    close(h, rh, tol(th, rh, "f32"), "h")
    guard = torch.full((T + 64, D), 3.0).cuda()
    hg = torch.full((4 + 2, D), 3.0).cuda()
    mb.mb_gated_scan(*c, cu_seqlens=torch.tensor([600, 100, 650, 20, 400], dtype=torch.int32).cuda(), y=guard[32:32 + T], h_out=hg[1:5], **kw)
    torch.cuda.synchronize()
    assert bool((guard[:32] == 3).all()) and bool((guard[32 + T:] == 3).all()) and bool((hg[0] == 3).all()) and bool((hg[5] == 3).all())
    out = mb.mb_gated_scan_bwd(*c[:3], d["dy"].cuda(), c[3], cu_seqlens=torch.tensor([600, 100, 650, 20, 400], dtype=torch.int32).cuda(),
                               dx=guard[32:32 + T], **kw)
    torch.cuda.synchronize()
    assert out[0].data_ptr() == guard[32].data_ptr() and bool((guard[:32] == 3).all()) and bool((guard[32 + T:] == 3).all())


def test_no_sequences_and_no_tokens():
    D = 20
    d = make(13, 100, D, "bf16", 3)
    none = torch.zeros(1, dtype=torch.int32).cuda()
    c = [d[k].cuda() for k in ("x", "a_gate", "decay", "x_gate")]
    y, h = mb.mb_gated_scan(*c, cu_seqlens=none, y=torch.full((100, D), 2.0, dtype=torch.bfloat16).cuda())
    assert bool((y == 2).all()) and h.shape == (0, D)
    out = mb.mb_gated_scan_bwd(*c[:3], d["dy"].cuda(), c[3], cu_seqlens=none)
    assert all(bool((out[i] == 0).all()) for i in range(4)) and out[6].shape == (0, D)
    e = torch.empty(0, D, dtype=torch.bfloat16).cuda()
    cu = torch.zeros(4, dtype=torch.int32).cuda()
    y, h, st = mb.mb_gated_scan(e, e, c[2], e, cu_seqlens=cu, h0=d["h0"].cuda(), states=True)
    assert torch.equal(h.cpu(), d["h0"]) and y.shape == (0, D) and st.shape == (0, D)
    y, h = mb.mb_gated_scan(e, e, c[2], e, cu_seqlens=cu)
    assert bool((h == 0).all())
    out = mb.mb_gated_scan_bwd(e, e, c[2], e, e, cu_seqlens=cu, h0=d["h0"].cuda(), dh_out=d["dh"].cuda())
    assert torch.equal(out[6].cpu(), d["dh"]) and bool((out[3] == 0).all())
    b = torch.empty(3, 0, D, dtype=torch.bfloat16).cuda()
    y, h = mb.mb_gated_scan(b, b, c[2], b, h0=d["h0"].cuda())
    assert torch.equal(h.cpu(), d["h0"])
    h, y = torch.empty(0, D).cuda(), None
    assert mb.mb_gated_scan_step(e, e, c[2], h, e)[0].shape == (0, D)


@pytest.mark.parametrize("T", [90, 2500])
def test_graph_replays(T):
    """Captured and replayed with other work in between: the same as the eager call, every time."""
    D = 96
    d = make(61, T, D, "bf16", 1)
    c = {k: v.cuda() for k, v in d.items()}
    bias = dict(a_bias=c["a_bias"], x_bias=c["x_bias"], h0=c["h0"])
    x, a, g, dy = (c[k][None] for k in ("x", "a_gate", "x_gate", "dy"))

    def both():
        y, h, st = mb.mb_gated_scan(x, a, c["decay"], g, states=True, **bias)
        return (y, h, st) + mb.mb_gated_scan_bwd(x, a, c["decay"], dy, g, dh_out=c["dh"], states=st, **bias)

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


def test_on_another_stream_and_side_by_side():
    """Two calls at once, each on a stream and a workspace of its own."""
    D, T = 64, 3000
    ds = [make(70 + i, T, D, "bf16", 1) for i in range(2)]
    cs = [{k: v.cuda() for k, v in d.items()} for d in ds]
    run = lambda c: mb.mb_gated_scan(c["x"][None], c["a_gate"][None], c["decay"], c["x_gate"][None], h0=c["h0"])  # noqa: E731
    want = [[t.clone() for t in run(c)] for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = []
    for _ in range(3):
        for s, c in zip(streams, cs):
            with torch.cuda.stream(s):
                got.append(run(c))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(o, want[i % 2]))


def test_long_cache_offsets():
    """Rows whose byte offsets pass 2^32: a wide stride, and a pool past it."""
    T, D, stride = 1100, 8, (1 << 22) - 8
    buf = torch.zeros(T * stride, dtype=torch.bfloat16, device="cuda")          # 9 GB
    d = make(81, T, D, "bf16", 1)
    views = [buf.view(T, stride)[:, i * D:(i + 1) * D] for i in range(3)]
    for v, k in zip(views, ("x", "a_gate", "x_gate")):
        v.copy_(d[k])
    n_slots = (1 << 30) // D + 5
    pool = torch.zeros(n_slots, D, device="cuda")
    slot = n_slots - 2
    pool[slot] = d["h0"][0].cuda()
    cu, sl = offsets([T]).cuda(), torch.tensor([slot], dtype=torch.int32).cuda()
    kw = dict(a_bias=d["a_bias"].cuda(), x_bias=d["x_bias"].cuda())
    y, _ = mb.mb_gated_scan(views[0], views[1], d["decay"].cuda(), views[2], cu_seqlens=cu, h0=pool, slots=sl, **kw)
    ry, rh, _, ty, th, _ = gf.scan(*wide(d), [T], d["h0"].double())
    close(y, ry, tol(ty, ry, "bf16"), "y")
    close(pool[slot], rh[0], tol(th[0], rh[0], "f32"), "h")
    out = mb.mb_gated_scan_bwd(views[0], views[1], d["decay"].cuda(), d["dy"].cuda(), views[2], cu_seqlens=cu, h0=d["h0"].cuda(), **kw)
    ref, bound = gf.scan_bwd(*wide(d), [T], d["dy"].double(), d["h0"].double())
    close(out[0], ref["dx"], tol(bound["dx"], ref["dx"], "bf16"), "dx")
    close(out[3], ref["ddecay"], tol(bound["ddecay"], ref["ddecay"], "f32"), "ddecay")


@pytest.mark.parametrize("T", [100, 700])
def test_padded_offsets(T):
    """Offsets padded to many more sequences than there are, as a captured graph has them: the padded ones have no tokens, and
    no row in the pool or one of their own; without a pool every one's state is written."""
    D, lens = 70, [T - 40, 0, 40] + [0] * 1500
    n = len(lens)
    d = make(91, T, D, "bf16", n)
    c = [d[k].cuda() for k in ("x", "a_gate", "decay", "x_gate")]
    bias = dict(a_bias=d["a_bias"].cuda(), x_bias=d["x_bias"].cuda(), cu_seqlens=offsets(lens).cuda())
    ry, rh, _, ty, th, _ = gf.scan(*wide(d), lens, d["h0"].double())
    y, h = mb.mb_gated_scan(*c, h0=d["h0"].cuda(), **bias)
    close(y, ry, tol(ty, ry, "bf16"), "y")
    close(h, rh, tol(th, rh, "f32"), "h")
    assert torch.equal(h[3:].cpu(), d["h0"][3:]) and torch.equal(h[1].cpu(), d["h0"][1])
    y, h = mb.mb_gated_scan(*c, **bias)
    assert bool((h[3:] == 0).all()) and bool((h[1] == 0).all())
    slots = torch.full((n,), -1, dtype=torch.int32)
    slots[:3], slots[900] = torch.tensor([2, 5, 0], dtype=torch.int32), 7
    has = torch.ones(n, dtype=torch.bool)
    has[900] = has[1] = False
    pool = torch.randn(9, D, generator=torch.Generator().manual_seed(1))
    start = torch.stack([pool[2], torch.zeros(D), pool[0]] + [torch.zeros(D)] * 1500).double()
    got = pool.clone().cuda()
    y, _ = mb.mb_gated_scan(*c, h0=got, slots=slots.cuda(), has_h0=has.cuda(), **bias)
    ry, rh, _, ty, th, _ = gf.scan(*wide(d), lens, start)
    close(y, ry, tol(ty, ry, "bf16"), "y")
    for s, row in ((0, 2), (2, 0)):
        close(got[row], rh[s], tol(th[s], rh[s], "f32"), "slot")
    assert bool((got[7] == 0).all()) and bool((got[5] == 0).all())
    for row in (1, 3, 4, 6, 8):
        assert torch.equal(got[row].cpu(), pool[row])
    out = mb.mb_gated_scan_bwd(*c[:3], d["dy"].cuda(), c[3], h0=d["h0"].cuda(), dh_out=d["dh"].cuda(), **bias)
    ref, bound = gf.scan_bwd(*wide(d), lens, d["dy"].double(), d["h0"].double(), d["dh"].double())
    for name, o in zip(("dx", "da_gate", "dx_gate", "ddecay", "da_bias", "dx_bias", "dh0"), out):
        close(o, ref[name], tol(bound[name], ref[name], "bf16" if o.dtype == torch.bfloat16 else "f32"), name)
    assert torch.equal(out[6][3:].cpu(), d["dh"][3:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("head,tail,D", [(20, 100, 64), (150, 300, 33), (64, 128, 6), (1000, 1, 64)])
def test_tokens_of_no_sequence(head, tail, D, dtype):
    """Many tokens in front of the first and behind the last sequence, whole tiles of them and parts of one, NaN in all that is theirs:
    the gradients are those of the sequences, and zero outside."""
    lens = [100, 37]
    n, T = len(lens), sum([100, 37])
    d = make(101, T, D, dtype, n)
    wrap = lambda t, v: torch.cat([torch.full((head, D), v, dtype=t.dtype), t, torch.full((tail, D), v, dtype=t.dtype)]).cuda()  # noqa: E731
    ins = [wrap(d["x"], float("nan")), wrap(d["a_gate"], float("nan")), d["decay"].cuda()]
    g, dy = wrap(d["x_gate"], float("nan")), wrap(d["dy"], float("nan"))
    kw = dict(a_bias=d["a_bias"].cuda(), x_bias=d["x_bias"].cuda(), cu_seqlens=(offsets(lens) + head).int().cuda(), h0=d["h0"].cuda())
    y, h, kept = mb.mb_gated_scan(*ins, g, y=wrap(torch.zeros_like(d["x"]), 7.0), states=True, **kw)
    ry, rh, _, ty, th, _ = gf.scan(*wide(d), lens, d["h0"].double())
    assert bool((y[:head] == 7.0).all()) and bool((y[head + T:] == 7.0).all())
    close(y[head:head + T], ry, tol(ty, ry, dtype), "y")
    close(h, rh, tol(th, rh, "f32"), "h")
    ref, bound = gf.scan_bwd(*wide(d), lens, d["dy"].double(), d["h0"].double(), d["dh"].double())
    for filled in (float("nan"), 3.0):
        kept[:head // 64], kept[-(-(head + T) // 64):] = filled, filled
        for bad in (g, dy, ins[0], ins[1]):
            bad[:head], bad[head + T:] = filled, filled
        for states in (None, kept):
            out = mb.mb_gated_scan_bwd(*ins, dy, g, dh_out=d["dh"].cuda(), states=states, **kw)
            for name, got in zip(("dx", "da_gate", "dx_gate", "ddecay", "da_bias", "dx_bias", "dh0"), out):
                if name in ("dx", "da_gate", "dx_gate"):
                    assert bool((got[:head] == 0).all()) and bool((got[head + T:] == 0).all()), name
                    got = got[head:head + T]
                close(got, ref[name], tol(bound[name], ref[name], dtype if got.dtype == DT[dtype] else "f32"), name)
    # a state that is not finite at the end of the last sequence
    ins[0][head + T - 1, 0] = float("nan")
    out = mb.mb_gated_scan_bwd(*ins, dy, g, dh_out=d["dh"].cuda(), **kw)
    for got in out[:3]:
        assert bool((got[:head] == 0).all()) and bool((got[head + T:] == 0).all())


# tiles hold 128 tokens forward and 64 back, groups 16 tiles, groups of groups 256: sequences that begin, and end, in a group's
# last tile, on its border, right behind it, and go on over many
LONG = [[70001], [1925, 30000, 1000, 3000, 33000], [2048, 32768 - 2048, 1, 2047, 16384], [2047, 1, 14331, 16389, 20], [1900, 200, 62, 30600, 70, 34000]]


@pytest.mark.parametrize("copies", [1, 131], ids=["few", "many"])
@pytest.mark.parametrize("lens", LONG, ids=lambda v: "-".join(map(str, v)))
def test_many_tiles(lens, copies):
    """Three channels, once and many times over (few and many columns of tiles hand on in different ways)."""
    D, T, n = 3, sum(lens), len(lens)
    d = make(111, T, D, "f32", n, decay="slow")
    c = {k: v.cuda().repeat(*[1] * (v.dim() - 1), copies) for k, v in d.items()}

    def one(t, name):
        t = t.reshape(*t.shape[:-1], copies, D)
        assert torch.equal(t, t[..., :1, :].expand_as(t)), name
        return t[..., 0, :]

    kw = dict(a_bias=c["a_bias"], x_bias=c["x_bias"], cu_seqlens=offsets(lens).cuda(), h0=c["h0"])
    y, h, kept = mb.mb_gated_scan(c["x"], c["a_gate"], c["decay"], c["x_gate"], states=True, **kw)
    ry, rh, _, ty, th, _ = gf.scan(*wide(d), lens, d["h0"].double())
    close(one(y, "y"), ry, tol(ty, ry, "f32"), "y")
    close(one(h, "h"), rh, tol(th, rh, "f32"), "h")
    ref, bound = gf.scan_bwd(*wide(d), lens, d["dy"].double(), d["h0"].double(), d["dh"].double())
    out = mb.mb_gated_scan_bwd(c["x"], c["a_gate"], c["decay"], c["dy"], c["x_gate"], dh_out=c["dh"], states=kept, **kw)
    for name, got in zip(("dx", "da_gate", "dx_gate", "ddecay", "da_bias", "dx_bias", "dh0"), out):
        close(one(got, name), ref[name], tol(bound[name], ref[name], "f32"), name)
