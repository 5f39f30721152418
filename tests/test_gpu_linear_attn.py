"""GPU: linear attention with a decay per head (chunked form, single tokens, backward) through
the C ABI against the float64 recurrences of tests/layer_forms.py.

Bounds, counted in u = 2^-24 (half a step of fp32) and h = 2^-8 (of bf16).  M is the same
result computed from absolute values: the sum of the magnitudes of everything added up.
* fp32: products and sums of one output pass through at most Dk + 64 additions, the carry once a
  chunk (two roundings each), and weights whose exponent x = n log2(lambda) is off by 2^-23 |x|
  (weights beyond x = 64 are below 2^-64): (2 Dk + 400 + 8 chunks) u M.
* bf16: the fp32 bound, one rounding of the masked scores and one of the state's copy (each
  term at most h of its magnitude, the two sets disjoint: h M) and one of the output (h |o|).
* states are fp32 in both (three bf16 pieces leave 2^-24 of a weighted value): the fp32 bound."""
import pytest
import torch

import layer_forms as lf
import selective_state_space_amd as mb
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
F64, U, HB = torch.float64, 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def decays(H, kind="mixed"):
    if kind == "mixed":
        return -torch.exp2(-8.0 * (torch.arange(H) + 1) / H).float()
    return {"none": torch.zeros(H), "strong": torch.full((H,), -20.0), "forget": torch.full((H,), float("-inf"))}[kind]


def inputs(seed, T, H, G, Dk, Dv, dtype, n, with_do=False):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s, d=DT[dtype]: torch.randn(*s, generator=g).to(d)
    d = dict(q=rn(T, H, Dk), k=rn(T, G, Dk), v=rn(T, G, Dv), h0=rn(n, H, Dk, Dv, d=torch.float32))
    if with_do:
        d.update(do=rn(T, H, Dv), dh=rn(n, H, Dk, Dv, d=torch.float32))
    return d


def bound(dtype, Dk, lens, M, ref):
    K = 2 * Dk + 400 + 8 * (max(lens, default=0) // 64 + 1)
    b = K * U * M
    return b + HB * (M + ref.abs()) if dtype == "bf16" else b


def close(got, ref, tol, what):
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), what + ": not finite"
    bad = (got - ref).abs() > tol
    assert not bool(bad.any()), "%s: %d of %d outside the bound, worst %.3g of it at %s" % (
        what, int(bad.sum()), bad.numel(), float(((got - ref).abs() / tol.clamp(min=1e-300)).max()), bad.nonzero()[0].tolist())


def reference(d, ld, scale, lens, h0):
    D = {k: t.double() for k, t in d.items()}
    h = None if h0 is None else h0.double()
    o, hs = lf.attn(D["q"], D["k"], D["v"], ld, scale, lens, h)
    Mo, Mh = lf.attn(D["q"].abs(), D["k"].abs(), D["v"].abs(), ld, abs(scale), lens, None if h is None else h.abs())
    return o, hs, Mo, Mh


def check_forward(o, h, d, ld, scale, lens, dtype, h0):
    ro, rh, Mo, Mh = reference(d, ld, scale, lens, h0)
    n = sum(lens)
    Dk = d["q"].shape[2]
    close(o.reshape(-1, *o.shape[-2:])[:n], ro[:n], bound(dtype, Dk, lens, Mo, ro)[:n], "o")
    close(h, rh, bound("f32", Dk, lens, Mh, rh), "h")


CASES = [  # lens (packed) or (n, L), H, G, Dk, Dv, decay
    ((1, 1), 1, 1, 16, 16, "mixed"), ((2, 63), 2, 1, 16, 20, "mixed"), ((1, 64), 3, 3, 64, 64, "none"),
    ((2, 65), 4, 2, 128, 64, "mixed"), ((1, 257), 2, 2, 40, 128, "mixed"), ((1, 130), 2, 2, 1, 1, "mixed"),
    ((1, 700), 2, 1, 64, 72, "mixed"),           # several segments, ragged end, two column tiles
    ((2, 1024), 1, 1, 128, 128, "none"),         # whole segments
    ((1, 300), 2, 2, 24, 100, "strong"), ((1, 300), 2, 2, 17, 33, "forget"),
    ([5, 0, 1, 64, 0, 200, 63], 4, 2, 64, 64, "mixed"), ([0, 0], 2, 2, 16, 16, "mixed"),
    ([700, 3, 0, 600, 1], 2, 1, 128, 64, "mixed"), ([1] * 300, 1, 1, 16, 16, "none"),
    ([1100, 3, 0, 600, 1], 2, 1, 128, 64, "mixed"), ([2] * 300 + [900] + [1] * 40, 2, 2, 16, 32, "mixed"),
    ((1, 1100), 2, 2, 128, 72, "mixed"), ((3, 520), 3, 3, 20, 40, "none"), ([0, 900, 0], 2, 2, 40, 24, "mixed"), ([256, 512, 257], 1, 1, 64, 20, "none")]


def _id(c):
    return "-".join(str(x) for x in c).replace(" ", "") if len(str(c[0])) < 40 else "many-" + "-".join(map(str, c[1:]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=_id)
def test_forward(case, dtype):
    spec, H, G, Dk, Dv, kind = case
    packed = isinstance(spec, list)
    lens = spec if packed else [spec[1]] * spec[0]
    T, n, ld = sum(lens), len(lens), decays(H, kind)
    d = inputs(7, T, H, G, Dk, Dv, dtype, n)
    q, k, v = (d[x].cuda() for x in "qkv")
    if packed:
        cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32).cuda()
    else:
        q, k, v = (t.view(*spec, *t.shape[1:]) for t in (q, k, v))
        cu = None
    for h0 in (None, d["h0"]):
        o, h = mb.mb_linear_attn(q, k, v, ld.cuda(), cu_seqlens=cu, h0=None if h0 is None else h0.cuda())
        assert o.dtype == q.dtype and o.shape == q.shape[:-1] + (Dv,)
        check_forward(o, h, d, ld, Dk ** -0.5, lens, dtype, h0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 1])
def test_forward_views_slots_and_tail(dtype, off):
    """Columns of one fused projection (also from an unaligned start), states in scattered slots of a
    pool, some sequences fresh, one without a slot, and rows behind the last sequence."""
    lens, H, G, Dk, Dv, tail = [70, 1, 0, 300, 65], 4, 2, 64, 32, 9
    n, T = len(lens), sum(lens)
    d = inputs(9, T, H, G, Dk, Dv, dtype, n)
    ld, width = decays(H), H * Dk + G * (Dk + Dv)
    wide = torch.full((T + tail, width + 8 + off), float("nan"), dtype=DT[dtype])
    cols = torch.cat([d["q"].flatten(1), d["k"].flatten(1), d["v"].flatten(1)], 1)
    wide[:T, off:off + width] = cols
    wide = wide.cuda()
    q, k, v = wide[:, off:off + width].split([H * Dk, G * Dk, G * Dv], 1)
    q, k, v = q.unflatten(1, (H, Dk)), k.unflatten(1, (G, Dk)), v.unflatten(1, (G, Dv))
    cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32).cuda()
    slots = torch.tensor([6, 0, 3, -1, 5], dtype=torch.int32)
    has = torch.tensor([1, 0, 1, 1, 0], dtype=torch.uint8)
    pool = torch.randn(8, H, Dk, Dv, generator=torch.Generator().manual_seed(3))
    start = torch.stack([pool[s] if s >= 0 and f else torch.zeros(H, Dk, Dv) for s, f in zip(slots.tolist(), has.tolist())])
    got = pool.clone().cuda()
    o = torch.full((T + tail, H, Dv), 7.0, dtype=DT[dtype]).cuda()
    o2, h2 = mb.mb_linear_attn(q, k, v, ld.cuda(), scale=0.3, cu_seqlens=cu, h0=got, has_h0=has.cuda(), slots=slots.cuda(), o=o)
    assert o2 is o and h2 is got
    assert bool((o[T:] == 7.0).all()), "rows behind the last sequence were written"
    ro, rh, Mo, Mh = reference(d, ld, 0.3, lens, start)
    close(o[:T], ro, bound(dtype, Dk, lens, Mo, ro), "o")
    for s, slot in enumerate(slots.tolist()):
        if slot >= 0:
            close(got[slot], rh[s], bound("f32", Dk, lens, Mh[s], rh[s]), "slot %d" % slot)
    for slot in (1, 2, 4, 7):
        assert torch.equal(got[slot].cpu(), pool[slot]), "an unnamed slot was written"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward_split_chains(dtype):
    """A sequence in two calls, the state handed on in place, equals one call to rounding."""
    L, a, H, Dk, Dv = 400, 173, 2, 64, 64
    d = inputs(11, L, H, H, Dk, Dv, dtype, 1)
    ld = decays(H)
    q, k, v = (d[x].cuda().view(1, L, H, -1) for x in "qkv")
    h = torch.zeros(1, H, Dk, Dv).cuda()
    o1, h = mb.mb_linear_attn(q[:, :a].contiguous(), k[:, :a].contiguous(), v[:, :a].contiguous(), ld.cuda(), h0=h, h_out=h)
    o2, h = mb.mb_linear_attn(q[:, a:].contiguous(), k[:, a:].contiguous(), v[:, a:].contiguous(), ld.cuda(), h0=h, h_out=h)
    check_forward(torch.cat([o1, o2], 1), h, d, ld, Dk ** -0.5, [L], dtype, None)


@pytest.mark.parametrize("few", [True, False], ids=["looked through", "table"])
def test_long_sequences_among_short_ones(few):
    """Sequences of more segments than the walk composes, whose states are composed beforehand, first, last and in between;
    offsets in front of the first token and behind the last count as these."""
    short = [5] * (20 if few else 150)
    lens, H, Dk, Dv = [4400] + short + [4501] + short + [2500, 4200], 2, 64, 64
    T, n = sum(lens), len(lens)
    d = inputs(61, T, H, H, Dk, Dv, "bf16", n)
    ld = torch.tensor([-0.002, -0.3])
    cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32)
    cu[0], cu[-1] = -70_000, T + 70_000
    o, h = mb.mb_linear_attn(*(d[x].cuda() for x in "qkv"), ld.cuda(), cu_seqlens=cu.cuda(), h0=d["h0"].cuda())
    check_forward(o, h, d, ld, Dk ** -0.5, lens, "bf16", d["h0"])


def test_offsets_out_of_range_stay_inside():
    """Offsets that decrease or leave [0, T] are empty or cut sequences: nothing outside is touched."""
    T, H, D = 1100, 2, 16
    d = inputs(12, T, H, H, D, D, "f32", 4)
    cu = torch.tensor([-5, 300, 200, 1500, 2000], dtype=torch.int32).cuda()   # [0,300), empty, [300,1100), empty
    q, k, v = (d[x].cuda() for x in "qkv")
    o, h = mb.mb_linear_attn(q, k, v, decays(H).cuda(), cu_seqlens=cu, h0=d["h0"].cuda())
    ref = {x: d[x] for x in "qkv"}
    ro, rh, Mo, Mh = reference({**ref}, decays(H), D ** -0.5, [300, 0, 800, 0], d["h0"])
    close(o, ro, bound("f32", D, [800], Mo, ro), "o")
    close(h, rh, bound("f32", D, [800], Mh, rh), "h")


BWD = [((1, 1), 1, 1, 16, 16, "mixed"), ((2, 65), 4, 2, 64, 20, "mixed"), ((1, 300), 2, 2, 128, 64, "mixed"),
       ((1, 130), 2, 1, 17, 33, "none"), ((1, 700), 3, 1, 40, 128, "mixed"), ((1, 200), 2, 2, 16, 16, "forget"),
       ([5, 0, 1, 64, 200], 4, 2, 64, 64, "mixed"), ([700, 3, 0, 300], 2, 1, 128, 32, "mixed"),
       ((1, 1100), 2, 1, 72, 128, "mixed"), ([900, 0, 300, 1], 2, 2, 64, 100, "mixed"), ([1100, 130], 2, 1, 128, 64, "mixed"), ([0, 0], 1, 1, 16, 16, "mixed")]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", BWD, ids=_id)
def test_backward(case, dtype):
    spec, H, G, Dk, Dv, kind = case
    packed = isinstance(spec, list)
    lens = spec if packed else [spec[1]] * spec[0]
    tail = 5 if packed else 0
    T, n, ld, scale = sum(lens), len(lens), decays(H, kind), 0.4
    d = inputs(21, T + tail, H, G, Dk, Dv, dtype, n, with_do=True)
    c = {x: t.cuda() for x, t in d.items()}
    cu = None
    if packed:
        cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32).cuda()
    else:
        for x in ("q", "k", "v", "do"):
            c[x] = c[x].view(*spec, *c[x].shape[1:])
    D = {x: t.double() for x, t in d.items()}
    A = {x: t.abs() for x, t in D.items()}
    for states in (True, False):
        out = mb.mb_linear_attn_bwd(c["q"], c["k"], c["v"], ld.cuda(), c["do"], scale=scale, cu_seqlens=cu,
                                    h0=c["h0"] if states else None, dh_out=c["dh"] if states else None)
        h0, dh = (D["h0"], D["dh"]) if states else (None, None)
        ref = lf.attn_bwd(D["q"], D["k"], D["v"], ld, scale, lens, D["do"], h0, dh)
        mag = lf.attn_bwd(A["q"], A["k"], A["v"], ld, scale, lens, A["do"], *((A["h0"], A["dh"]) if states else (None, None)))
        rep = H // G
        for name, got, r, M in zip(("dq", "dk", "dv", "dh0"), out, ref, mag):
            tol = bound("f32" if name == "dh0" else dtype, max(Dk, Dv) + 4 * rep, lens, M, r)
            close(got.reshape(r.shape), r, tol, name)
        again = mb.mb_linear_attn_bwd(c["q"], c["k"], c["v"], ld.cuda(), c["do"], scale=scale, cu_seqlens=cu,
                                      h0=c["h0"] if states else None, dh_out=c["dh"] if states else None)
        assert all(torch.equal(a, b) for a, b in zip(out, again)), "two runs differ"


STEP = [(1, 16, 16, 128, 64), (5, 4, 2, 64, 64), (3, 2, 1, 40, 20), (70, 8, 8, 128, 128), (2, 3, 3, 17, 33), (1, 1, 1, 1, 1),
        (40, 16, 4, 24, 6)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", STEP, ids=lambda c: "x".join(map(str, c)))
def test_step(case, dtype):
    n, H, G, Dk, Dv = case
    d = inputs(31, n, H, G, Dk, Dv, dtype, n + 3)
    ld, pool = decays(H), d["h0"]
    slots = torch.randperm(n + 3, generator=torch.Generator().manual_seed(1))[:n].int()
    if n > 2:
        slots[1] = -1                              # a padding row
        slots[2] = n + 3                           # and one past the pool
    ok = [0 <= s < n + 3 for s in slots.tolist()]
    start = torch.stack([pool[s] if f else torch.zeros(H, Dk, Dv) for s, f in zip(slots.tolist(), ok)])
    ro, rh, Mo, Mh = reference(d, ld, 0.5, [1] * n, start)
    got = pool.clone().cuda()
    o, h = mb.mb_linear_attn_step(d["q"].cuda(), d["k"].cuda(), d["v"].cuda(), ld.cuda(), got, scale=0.5, slots=slots.cuda())
    assert h is got
    # one product per state value and one sum over the rows: the fp32 bound and the output's rounding
    tol = (Dk + 64) * U * Mo + (HB * ro.abs() if dtype == "bf16" else 0.0)
    close(o, ro, tol, "o")
    named = set()
    for i, (s, f) in enumerate(zip(slots.tolist(), ok)):
        if f:
            named.add(s)
            close(got[s], rh[i], 16 * U * Mh[i], "slot %d" % s)
    for s in range(n + 3):
        if s not in named:
            assert torch.equal(got[s].cpu(), pool[s])
    # contiguous states, into another tensor
    o2, h2 = mb.mb_linear_attn_step(d["q"].cuda(), d["k"].cuda(), d["v"].cuda(), ld.cuda(), start.cuda(), scale=0.5,
                                    h_out=torch.empty_like(start).cuda())
    assert torch.equal(o2, o)
    close(h2, rh, 16 * U * Mh, "h")


def test_step_continues_the_chunked_form():
    L, L0, H, Dk, Dv = 90, 77, 2, 64, 64
    d = inputs(41, L, H, H, Dk, Dv, "f32", 1)
    ld = decays(H).cuda()
    q, k, v = (d[x].cuda().view(1, L, H, -1) for x in "qkv")
    o, h = mb.mb_linear_attn(q[:, :L0].contiguous(), k[:, :L0].contiguous(), v[:, :L0].contiguous(), ld)
    rows = [o]
    for t in range(L0, L):
        y, h = mb.mb_linear_attn_step(q[:, t].contiguous(), k[:, t].contiguous(), v[:, t].contiguous(), ld, h)
        rows.append(y[:, None])
    check_forward(torch.cat(rows, 1), h, d, decays(H), Dk ** -0.5, [L], "f32", None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("widths", [(64, 64), (100, 52), (33, 127)], ids=str)
@pytest.mark.parametrize("off", [1, 2, 3])
def test_backward_of_views_at_any_address(off, widths, dtype):
    """q, k and v as columns of one buffer that starts at an odd element, its rows longer than these by an odd number."""
    (Dk, Dv), H, lens = widths, 2, [70, 1, 300]
    T, n, ld = sum(lens), len(lens), decays(H)
    d = inputs(71, T, H, H, Dk, Dv, dtype, n, with_do=True)
    wide = H * (2 * Dk + Dv) + off
    buf = torch.full((off + T * wide,), 9.0, dtype=DT[dtype]).cuda()
    rows = buf[off:].view(T, wide)
    at, c = 0, {}
    for x, D in (("q", Dk), ("k", Dk), ("v", Dv)):
        rows[:, at:at + H * D] = d[x].reshape(T, H * D).cuda()
        c[x] = rows[:, at:at + H * D].unflatten(1, (H, D))
        at += H * D
    cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32).cuda()
    do = torch.empty(T * H * Dv + off, dtype=DT[dtype], device="cuda")[off:].view(T, H, Dv).copy_(d["do"])
    out = mb.mb_linear_attn_bwd(c["q"], c["k"], c["v"], ld.cuda(), do, scale=0.3, cu_seqlens=cu)
    D64 = {x: t.double() for x, t in d.items()}
    A = {x: t.abs() for x, t in D64.items()}
    ref = lf.attn_bwd(D64["q"], D64["k"], D64["v"], ld, 0.3, lens, D64["do"])
    mag = lf.attn_bwd(A["q"], A["k"], A["v"], ld, 0.3, lens, A["do"])
    for name, got, r, M in zip(("dq", "dk", "dv"), out, ref, mag):
        close(got, r, bound(dtype, max(Dk, Dv) + 4, lens, M, r), name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_later_tokens_and_other_sequences_do_not_reach_back(dtype):
    """Infinite values and NaN keys, in the middle of a chunk: earlier tokens and the other sequences as without."""
    lens, H, D = [100, 200, 30], 2, 64
    T, bad = sum(lens), 100 + 140
    cu = torch.tensor([0, 100, 300, 330], dtype=torch.int32).cuda()
    d = inputs(51, T, H, H, D, D, dtype, 3)
    ld = decays(H)
    ro, rh, Mo, Mh = reference(d, ld, D ** -0.5, lens, None)
    tol = bound(dtype, D, lens, Mo, ro)
    for what, value in (("v", float("inf")), ("v", float("nan")), ("k", float("nan")), ("q", float("nan"))):
        c = {x: d[x].clone() for x in "qkv"}
        c[what][bad, :, 5] = value
        o, h = mb.mb_linear_attn(*(c[x].cuda() for x in "qkv"), ld.cuda(), cu_seqlens=cu)
        keep = [i for i in range(T) if i < bad or i >= 300 or (what == "q" and i != bad)]
        close(o[keep], ro[keep], tol[keep], "o beside %s = %s" % (what, value))
        close(h[[0, 2]], rh[[0, 2]], bound("f32", D, lens, Mh, rh)[[0, 2]], "h")
        if what == "q":
            assert bool(torch.isnan(o[bad]).all())
        else:
            hit = o[bad:300, :, 5] if what == "v" else o[bad:300]
            assert not bool(torch.isfinite(hit[0]).any()) and not bool(torch.isfinite(h[1]).all())
            if what == "v":
                rest = [i for i in range(D) if i != 5]
                close(o[:, :, rest], ro[:, :, rest], tol[:, :, rest], "other columns")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_of_later_tokens_alone(dtype):
    """A NaN in do reaches dq of its own token and dk, dv up to it, nothing behind it and no other sequence."""
    lens, H, D = [40, 200, 30], 2, 64
    T, bad = sum(lens), 40 + 100
    cu = torch.tensor([0, 40, 240, 270], dtype=torch.int32).cuda()
    d = inputs(52, T, H, H, D, D, dtype, 3, with_do=True)
    ld = decays(H)
    D64 = {x: t.double() for x, t in d.items()}
    A = {x: t.abs() for x, t in D64.items()}
    ref = lf.attn_bwd(D64["q"], D64["k"], D64["v"], ld, 0.3, lens, D64["do"])
    mag = lf.attn_bwd(A["q"], A["k"], A["v"], ld, 0.3, lens, A["do"])
    d["do"][bad, :, 3] = float("nan")
    out = mb.mb_linear_attn_bwd(*(d[x].cuda() for x in "qkv"), ld.cuda(), d["do"].cuda(), scale=0.3, cu_seqlens=cu)
    keep_q = [i for i in range(T) if i != bad]
    keep_kv = [i for i in range(T) if i < 40 or i > bad]
    for name, got, r, M, keep in (("dq", out[0], ref[0], mag[0], keep_q), ("dk", out[1], ref[1], mag[1], keep_kv), ("dv", out[2], ref[2], mag[2], keep_kv)):
        close(got[keep], r[keep], bound(dtype, D + 4, lens, M, r)[keep], name)
    assert bool(torch.isnan(out[0][bad]).all()) and bool(torch.isnan(out[1][40:bad + 1]).all())


def test_no_sequences_and_no_tokens():
    q = torch.randn(5, 2, 16).cuda()
    ld, cu = decays(2).cuda(), torch.tensor([3], dtype=torch.int32).cuda()
    o = torch.full_like(q, 7.0)
    o2, h = mb.mb_linear_attn(q, q, q, ld, cu_seqlens=cu, o=o)
    assert bool((o2 == 7.0).all()) and h.shape == (0, 2, 16, 16)
    for g in mb.mb_linear_attn_bwd(q, q, q, ld, q, cu_seqlens=cu)[:3]:
        assert bool((g == 0).all())
    e = torch.empty(3, 0, 2, 16).cuda()
    h0 = torch.randn(3, 2, 16, 16).cuda()
    o, h = mb.mb_linear_attn(e, e, e, ld, h0=h0)
    assert o.shape == e.shape and torch.equal(h, h0)
    assert torch.equal(mb.mb_linear_attn_bwd(e, e, e, ld, e, dh_out=h0)[3], h0)
    o, h = mb.mb_linear_attn(e[:0], e[:0], e[:0], ld)
    assert o.shape[0] == 0 and h.shape[0] == 0


def test_states_behind_two_to_the_31_elements():
    """A pool of more than 2^31 values: the last slots, chunked form and step."""
    H, Dk, Dv, n_slots = 16, 128, 128, 8300
    pool = torch.empty(n_slots, H, Dk, Dv, device="cuda")
    assert pool.numel() > 2 ** 31
    slots = torch.tensor([n_slots - 1, n_slots - 3], dtype=torch.int32)
    d = inputs(53, 140, H, H, Dk, Dv, "bf16", 2)
    for s, h in zip(slots.tolist(), d["h0"]):
        pool[s] = h.cuda()
    cu = torch.tensor([0, 70, 140], dtype=torch.int32).cuda()
    ld, c = decays(H), {x: d[x].cuda() for x in "qkv"}
    o, _ = mb.mb_linear_attn(c["q"], c["k"], c["v"], ld.cuda(), cu_seqlens=cu, h0=pool, slots=slots.cuda())
    ro, rh, Mo, Mh = reference(d, ld, Dk ** -0.5, [70, 70], d["h0"])
    close(o, ro, bound("bf16", Dk, [70], Mo, ro), "o")
    close(pool[slots.long().cuda()], rh, bound("f32", Dk, [70], Mh, rh), "h")
    start = pool[slots.long().cuda()].cpu()
    one = {x: d[x][:2] for x in "qkv"}
    o, _ = mb.mb_linear_attn_step(*(one[x].cuda() for x in "qkv"), ld.cuda(), pool, slots=slots.cuda())
    ro, rh, Mo, Mh = reference(one, ld, Dk ** -0.5, [1, 1], start)
    close(o, ro, (Dk + 64) * U * Mo + HB * ro.abs(), "o")
    close(pool[slots.long().cuda()], rh, 16 * U * Mh, "h")


def _graph(fn):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fn()
    return g, out


def test_captured_and_replayed():
    """Forward, step and backward in one graph, replayed on new inputs with eager work in between."""
    lens, H, G, Dk, Dv = [600, 1, 700], 2, 1, 64, 64
    T, n = sum(lens), len(lens)
    cu = torch.tensor([0, 600, 601, 1301], dtype=torch.int32).cuda()
    d = {x: t.cuda() for x, t in inputs(61, T, H, G, Dk, Dv, "bf16", n, with_do=True).items()}
    ld, one = decays(H).cuda(), [t[:n].clone() for t in (d["q"], d["k"], d["v"])]

    def fn():
        o, h = mb.mb_linear_attn(d["q"], d["k"], d["v"], ld, cu_seqlens=cu, h0=d["h0"])
        y, h = mb.mb_linear_attn_step(*one, ld, h)
        return (o, h, y) + mb.mb_linear_attn_bwd(d["q"], d["k"], d["v"], ld, d["do"], cu_seqlens=cu, h0=d["h0"], dh_out=d["dh"])

    g, out = _graph(fn)
    for r in range(4):
        new = inputs(70 + r, T, H, G, Dk, Dv, "bf16", n, with_do=True)
        for x in d:
            d[x].copy_(new[x])
        cu.copy_(torch.tensor([[0, 600, 601, 1301], [0, 0, 1300, 1301], [0, 1, 2, 1301], [0, 650, 1300, 1301]][r], dtype=torch.int32))
        want = fn()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), "replay %d differs from the eager call" % r


def test_other_stream():
    d = {x: t.cuda() for x, t in inputs(81, 500, 2, 2, 64, 64, "bf16", 1).items()}
    q, k, v = (d[x].view(1, 500, 2, 64) for x in "qkv")
    ld = decays(2).cuda()
    want = mb.mb_linear_attn(q, k, v, ld)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = mb.mb_linear_attn(q, k, v, ld)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
