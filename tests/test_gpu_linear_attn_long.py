"""GPU: linear attention, forward and backward, where sequences have more segments than a walk composes (their states
are composed beforehand), where the segments come from a table, and where every token's share is visible.

All inputs are positive, so that nothing cancels: a result is the sum of the magnitudes M that its bound is counted in (see
tests/test_gpu_linear_attn.py).  With a decay of e^-0.05 a token weighs a twentieth of what it reaches first, six times the
bf16 bound (2^-8 of M twice); with e^-0.0005 a segment of 256 tokens weighs an eighth of what enters the next one."""
import pytest
import torch

import layer_forms as lf
import selective_state_space_amd as mb
from gpu_util import require_gpu
from test_gpu_linear_attn import DT, bound, close

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def positive(seed, T, H, G, Dk, Dv, dtype, n):
    g = torch.Generator().manual_seed(seed)
    u = lambda *s, d=DT[dtype]: (0.5 + torch.rand(*s, generator=g)).to(d)
    f = torch.float32
    return dict(q=u(T, H, Dk), k=u(T, G, Dk), v=u(T, G, Dv), do=u(T, H, Dv), h0=20 * u(n, H, Dk, Dv, d=f), dh=20 * u(n, H, Dk, Dv, d=f))


MANY = [5] * 150 + [4500] + [3] * 150 + [0, 600]      # the table, and a sequence of more than 16 segments
CASES = [  # lens (packed) or (n, L), H, G, Dk, Dv
    ((1, 4500), 2, 2, 64, 64), ((1, 4500), 2, 1, 128, 72), ((1, 4417), 1, 1, 40, 128), ((2, 4500), 2, 2, 128, 128), ((1, 4500), 2, 2, 128, 64),
    ([7, 4500, 0, 300], 2, 2, 64, 40), ([4500, 7], 2, 1, 128, 128), ([300, 4400], 2, 2, 20, 100),
    (MANY, 2, 2, 64, 64), (MANY, 2, 2, 128, 128), (MANY, 2, 1, 128, 32), (MANY, 2, 2, 33, 100)]


def _id(c):
    return "-".join(map(str, ("many" if c[0] is MANY else c[0],) + c[1:])).replace(" ", "")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=_id)
def test_long_forward_and_backward(case, dtype):
    spec, H, G, Dk, Dv = case
    packed = isinstance(spec, list)
    lens = spec if packed else [spec[1]] * spec[0]
    T, n, scale = sum(lens), len(lens), Dk ** -0.5
    ld = torch.tensor([-0.05, -0.0005])[:H]
    d = positive(91, T, H, G, Dk, Dv, dtype, n)
    c, cu = {x: t.cuda() for x, t in d.items()}, None
    if packed:
        cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32).cuda()
    else:
        c.update({x: c[x].view(*spec, *c[x].shape[1:]) for x in ("q", "k", "v", "do")})
    D = {x: t.double() for x, t in d.items()}
    ro, rh = lf.attn(D["q"], D["k"], D["v"], ld, scale, lens, D["h0"])
    o, h = mb.mb_linear_attn(c["q"], c["k"], c["v"], ld.cuda(), cu_seqlens=cu, h0=c["h0"])
    close(o.reshape(ro.shape), ro, bound(dtype, Dk, lens, ro, ro), "o")
    close(h, rh, bound("f32", Dk, lens, rh, rh), "h")
    ref = lf.attn_bwd(D["q"], D["k"], D["v"], ld, scale, lens, D["do"], D["h0"], D["dh"])
    call = lambda: mb.mb_linear_attn_bwd(c["q"], c["k"], c["v"], ld.cuda(), c["do"], cu_seqlens=cu, h0=c["h0"], dh_out=c["dh"])
    out = call()
    for name, got, r in zip(("dq", "dk", "dv", "dh0"), out, ref):
        close(got.reshape(r.shape), r, bound("f32" if name == "dh0" else dtype, max(Dk, Dv) + 4 * (H // G), lens, r, r), name)
    assert all(torch.equal(a, b) for a, b in zip(out, call())), "two runs differ"
    o2, h2 = mb.mb_linear_attn(c["q"], c["k"], c["v"], ld.cuda(), cu_seqlens=cu, h0=c["h0"])
    assert torch.equal(o, o2) and torch.equal(h, h2), "two runs differ"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_in_place_in_a_pool(dtype):
    """The states' composition beforehand with slots: h_out is h0, and one sequence has no slot."""
    lens, H, Dk, Dv = [4500, 3, 4400, 20], 2, 64, 72
    T, n, ld = sum(lens), len(lens), torch.tensor([-0.05, -0.0005])
    d = positive(92, T, H, H, Dk, Dv, dtype, 6)
    slots, has = torch.tensor([4, 1, -1, 0], dtype=torch.int32), torch.tensor([True, False, True, True])
    start = torch.stack([d["h0"][s] if s >= 0 and f else torch.zeros(H, Dk, Dv) for s, f in zip(slots.tolist(), has.tolist())])
    cu = torch.tensor([0, 4500, 4503, 8903, 8923], dtype=torch.int32).cuda()
    pool = d["h0"].clone().cuda()
    o, _ = mb.mb_linear_attn(*(d[x].cuda() for x in "qkv"), ld.cuda(), cu_seqlens=cu, h0=pool, has_h0=has.cuda(), slots=slots.cuda())
    ro, rh = lf.attn(*(d[x].double() for x in "qkv"), ld, Dk ** -0.5, lens, start.double())
    close(o, ro, bound(dtype, Dk, lens, ro, ro), "o")
    for s, slot in enumerate(slots.tolist()):
        if slot >= 0:
            close(pool[slot], rh[s], bound("f32", Dk, lens, rh[s], rh[s]), "slot %d" % slot)
    for slot in (2, 3, 5):
        assert torch.equal(pool[slot].cpu(), d["h0"][slot])


def test_long_captured_and_replayed():
    """A graph of the forward and the backward with a table and composed states, on other lengths each time."""
    n, T, H, D = 300, 5400, 2, 64
    ld = torch.tensor([-0.05, -0.0005]).cuda()
    c = {x: t.cuda() for x, t in positive(93, T, H, H, D, D, "bf16", n).items()}

    def offsets(r):
        g = torch.Generator().manual_seed(r)
        lens = torch.randint(0, 4, (n,), generator=g)
        lens[r * 70] = 0
        lens[r * 70] = T - int(lens.sum()) - 40 * r
        return torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).int()

    cu = offsets(0).cuda()

    def fn():
        return mb.mb_linear_attn(c["q"], c["k"], c["v"], ld, cu_seqlens=cu, h0=c["h0"], o=o) + \
            mb.mb_linear_attn_bwd(c["q"], c["k"], c["v"], ld, c["do"], cu_seqlens=cu, h0=c["h0"], dh_out=c["dh"])

    o = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fn()
    for r in range(4):
        cu.copy_(offsets(r))
        o.zero_()
        want = [t.clone() for t in fn()]
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), "replay %d differs from the eager call" % r
