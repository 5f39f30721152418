"""CPU: what the gated recurrence and the norm of queries and keys refuse, on the host and before anything is enqueued (no
pointer here is ever dereferenced), and what the binding takes."""
import ctypes

import pytest
import torch

import selective_state_space_amd as mb

OK, E_NULL, E_SHAPE, E_DTYPE, E_WS, E_HIP, E_ALIAS, E_ALIGN = range(8)
F32, BF16 = 0, 1
M = 1 << 28
INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(mb.lib_path()):
        from selective_state_space_amd import _build
        _build.build()
    return mb.load_library()


def p(x):
    return ctypes.c_void_p(x) if x else None


def scan(lib, x=M, a=2 * M, g=3 * M, dec=4 * M, ab=5 * M, xb=6 * M, cu=0, h0=0, has=0, slots=0, y=7 * M, h=8 * M, st=9 * M, n=2, T=600, D=64, ns=0,
         xs=64, as_=64, gs=64, dt=F32, ws=10 * M, nws=M):
    return lib.mb_gated_scan(p(x), p(a), p(g), p(dec), p(ab), p(xb), p(cu), p(h0), p(has), p(slots), p(y), p(h), p(st), n, T, D, ns, xs, as_, gs,
                             dt, p(ws), nws, None)


def test_gated_scan(lib):
    for dt in (2, -1):
        assert scan(lib, dt=dt) == E_DTYPE
    for kw in (dict(n=-1), dict(T=-1), dict(D=0), dict(T=601), dict(xs=63), dict(as_=1), dict(gs=63), dict(T=1 << 31), dict(n=(1 << 20) + 1),
               dict(xs=1 << 22), dict(D=1 << 22, xs=1 << 22, as_=1 << 22, gs=1 << 22), dict(slots=11 * M, ns=1 << 31), dict(ns=3), dict(slots=11 * M),
               dict(slots=11 * M, ns=-1), dict(T=(1 << 31) - 2, D=100000, xs=100000, as_=100000, gs=100000)):
        assert scan(lib, **kw) == E_SHAPE, kw
    for kw in (dict(x=0), dict(a=0), dict(dec=0), dict(y=0), dict(g=0)):            # x_bias without an x_gate
        assert scan(lib, **kw) == E_NULL, kw
    for kw in (dict(x=M + 2), dict(a=2 * M + 1), dict(g=3 * M + 1, dt=BF16), dict(dec=4 * M + 2), dict(ab=5 * M + 2), dict(xb=6 * M + 2), dict(cu=11 * M + 2),
               dict(h0=11 * M + 2), dict(slots=11 * M + 1, ns=4), dict(y=7 * M + 2), dict(h=8 * M + 2), dict(st=9 * M + 2)):
        assert scan(lib, **kw) == E_ALIGN, kw
    for kw in (dict(y=M), dict(y=2 * M + 64), dict(y=3 * M), dict(y=4 * M), dict(h=M), dict(h=7 * M), dict(h0=8 * M + 4), dict(st=M), dict(st=7 * M), dict(st=8 * M),
               dict(slots=8 * M, ns=4), dict(cu=7 * M), dict(has=9 * M, h0=11 * M)):
        assert scan(lib, **kw) == E_ALIAS, kw
    need = mb.mb_workspace_size(mb.MB_OP_GATED_SCAN, 2, 600, 64, 1, 1, 1)
    if need:
        for kw in (dict(nws=need - 1), dict(ws=0), dict(ws=10 * M + 64)):
            assert scan(lib, **kw) == E_WS, kw
        for kw in (dict(ws=M), dict(ws=7 * M), dict(ws=9 * M)):
            assert scan(lib, **kw) == E_ALIAS, kw
    assert scan(lib, n=0) == OK
    assert mb.mb_workspace_size(mb.MB_OP_GATED_SCAN, 2, 600, 0, 1, 1, 1) == 0


def step(lib, x=M, a=2 * M, g=3 * M, dec=4 * M, ab=5 * M, xb=6 * M, slots=0, hi=8 * M, ho=8 * M, y=7 * M, n=5, D=64, ns=0, xs=64, as_=64, gs=64, dt=F32):
    return lib.mb_gated_scan_step(p(x), p(a), p(g), p(dec), p(ab), p(xb), p(slots), p(hi), p(ho), p(y), n, D, ns, xs, as_, gs, dt, None)


def test_gated_scan_step(lib):
    assert step(lib, dt=2) == E_DTYPE
    for kw in (dict(n=-1), dict(D=0), dict(xs=63), dict(ns=1), dict(slots=9 * M), dict(n=(1 << 20) + 1)):
        assert step(lib, **kw) == E_SHAPE, kw
    for kw in (dict(x=0), dict(a=0), dict(dec=0), dict(ho=0), dict(y=0), dict(g=0)):
        assert step(lib, **kw) == E_NULL, kw
    for kw in (dict(ho=8 * M + 64), dict(y=M), dict(y=8 * M), dict(ho=3 * M), dict(slots=8 * M, ns=7)):
        assert step(lib, **kw) == E_ALIAS, kw
    for kw in (dict(hi=8 * M + 2), dict(x=M + 1), dict(y=7 * M + 1)):
        assert step(lib, **kw) == E_ALIGN, kw
    assert step(lib, n=0) == OK


def sbwd(lib, x=M, a=2 * M, g=3 * M, dec=4 * M, ab=5 * M, xb=6 * M, cu=0, h0=0, dy=7 * M, dh=0, st=0, dx=8 * M, da=9 * M, dg=10 * M, dd=11 * M, dab=12 * M,
         dxb=13 * M, dh0=14 * M, n=2, T=600, D=64, xs=64, as_=64, gs=64, dt=F32, ws=15 * M, nws=M):
    return lib.mb_gated_scan_bwd(p(x), p(a), p(g), p(dec), p(ab), p(xb), p(cu), p(h0), p(dy), p(dh), p(st), p(dx), p(da), p(dg), p(dd), p(dab), p(dxb), p(dh0),
                                 n, T, D, xs, as_, gs, dt, p(ws), nws, None)


def test_gated_scan_bwd(lib):
    assert sbwd(lib, dt=2) == E_DTYPE
    for kw in (dict(n=-1), dict(D=0), dict(T=601), dict(xs=63), dict(n=0)):
        assert sbwd(lib, **kw) == E_SHAPE, kw
    for kw in (dict(x=0), dict(a=0), dict(dec=0), dict(dy=0), dict(dx=0), dict(da=0), dict(dg=0), dict(g=0, xb=0), dict(g=0, xb=0, dg=0)):
        assert sbwd(lib, **kw) == E_NULL, kw
    for kw in (dict(dy=7 * M + 2), dict(dx=8 * M + 1), dict(dh=16 * M + 2), dict(st=16 * M + 2), dict(dd=11 * M + 1), dict(dh0=14 * M + 2)):
        assert sbwd(lib, **kw) == E_ALIGN, kw
    for kw in (dict(dx=M), dict(da=7 * M), dict(dg=8 * M), dict(dd=4 * M), dict(dab=11 * M), dict(dxb=6 * M), dict(dh=14 * M), dict(st=8 * M), dict(ws=8 * M),
               dict(ws=7 * M), dict(dh0=10 * M)):
        assert sbwd(lib, **kw) == E_ALIAS, kw
    need = mb.mb_workspace_size(mb.MB_OP_GATED_SCAN_BWD, 2, 600, 64, 1, 1, 1)
    assert need > 0
    for kw in (dict(nws=need - 1), dict(ws=0), dict(ws=15 * M + 64)):
        assert sbwd(lib, **kw) == E_WS, kw


def qk(lib, q=M, k=2 * M, wq=3 * M, wk=4 * M, f=5 * M, pos=6 * M, qo=7 * M, ko=8 * M, T=100, L=100, Hq=4, Hk=2, D=64, R=64, qs=256, ks=128, qos=256, kos=128,
       inter=0, eps=1e-5, dt=F32):
    return lib.mb_qk_norm_rope(p(q), p(k), p(wq), p(wk), p(f), p(pos), p(qo), p(ko), T, L, Hq, Hk, D, R, qs, ks, qos, kos, inter, eps, dt, None)


def test_qk_norm_rope(lib):
    assert qk(lib, dt=2) == E_DTYPE
    for kw in (dict(T=-1), dict(T=(1 << 30) + 1), dict(Hq=0), dict(Hk=-1), dict(Hq=4097, qs=1 << 21, qos=1 << 21), dict(D=0), dict(D=513, qs=4096, ks=4096, qos=4096, kos=4096),
               dict(R=63), dict(R=66), dict(R=-2), dict(qs=255), dict(ks=127), dict(qos=255), dict(kos=1), dict(qs=1 << 22), dict(pos=0, L=0), dict(eps=-1.0),
               dict(eps=INF), dict(eps=float("nan"))):
        assert qk(lib, **kw) == E_SHAPE, kw
    for kw in (dict(q=0), dict(k=0), dict(qo=0), dict(ko=0), dict(f=0)):
        assert qk(lib, **kw) == E_NULL, kw
    for kw in (dict(q=M + 2), dict(qo=7 * M + 1), dict(wq=3 * M + 2), dict(f=5 * M + 2), dict(pos=6 * M + 1), dict(k=2 * M + 1, dt=BF16)):
        assert qk(lib, **kw) == E_ALIGN, kw
    for kw in (dict(qo=M + 4), dict(qo=2 * M), dict(ko=M), dict(ko=7 * M), dict(qo=3 * M), dict(qo=M, qos=300), dict(qo=5 * M), dict(ko=6 * M),
               dict(qo=7 * M, qos=512, ko=7 * M + 1020, kos=512), dict(qo=7 * M, qos=512, ko=7 * M + 4 * 512 * 3 - 4, kos=512)):
        assert qk(lib, **kw) == E_ALIAS, kw
    assert qk(lib, T=0) == OK


def qbwd(lib, dqo=M, dko=2 * M, q=3 * M, k=4 * M, wq=5 * M, wk=6 * M, f=7 * M, pos=8 * M, dq=9 * M, dk=10 * M, dwq=11 * M, dwk=12 * M, T=100, L=100, Hq=4, Hk=2,
         D=64, R=64, qs=256, ks=128, inter=0, eps=1e-5, dt=F32, ws=13 * M, nws=M):
    return lib.mb_qk_norm_rope_bwd(p(dqo), p(dko), p(q), p(k), p(wq), p(wk), p(f), p(pos), p(dq), p(dk), p(dwq), p(dwk), T, L, Hq, Hk, D, R, qs, ks, inter, eps,
                                   dt, p(ws), nws, None)


def test_qk_norm_rope_bwd(lib):
    assert qbwd(lib, dt=5) == E_DTYPE
    for kw in (dict(T=-1), dict(D=513), dict(R=3), dict(qs=255), dict(pos=0, L=0), dict(eps=-1.0)):
        assert qbwd(lib, **kw) == E_SHAPE, kw
    for kw in (dict(dqo=0), dict(dko=0), dict(q=0), dict(k=0), dict(dq=0), dict(dk=0), dict(f=0)):
        assert qbwd(lib, **kw) == E_NULL, kw
    for kw in (dict(dq=M), dict(dk=4 * M), dict(dwq=5 * M), dict(dwk=11 * M), dict(dk=9 * M), dict(ws=9 * M), dict(ws=3 * M)):
        assert qbwd(lib, **kw) == E_ALIAS, kw
    for kw in (dict(dqo=M + 2), dict(dwq=11 * M + 2), dict(dk=10 * M + 1)):
        assert qbwd(lib, **kw) == E_ALIGN, kw
    need = mb.mb_workspace_size(mb.MB_OP_QK_NORM_ROPE_BWD, 100, 1, 4, 64, 2, 1)
    assert need > 0
    for kw in (dict(nws=need - 1), dict(ws=0), dict(ws=13 * M + 64)):
        assert qbwd(lib, **kw) == E_WS, kw


def test_binding_refuses_cpu_tensors_and_odd_calls():
    x, h = torch.zeros(2, 8), torch.zeros(2, 8)
    q = torch.zeros(3, 2, 8)
    for call in (lambda: mb.mb_gated_scan(x[None], x[None], x[0]), lambda: mb.mb_gated_scan_step(x, x, x[0], h), lambda: mb.mb_gated_scan_bwd(x[None], x[None], x[0], x[None]),
                 lambda: mb.mb_qk_norm_rope(q, q), lambda: mb.mb_qk_norm_rope_bwd(q, q, q, q)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_channel_strides():
    dev, f = torch.device("cpu"), torch.float32
    buf = torch.zeros(2, 5, 40)
    assert mb._channels(buf[..., 8:32], "x", (2, 5), 24, f, dev) == 40
    assert mb._channels(buf[0, :, :24], "x", (5,), 24, f, dev) == 40
    assert mb._channels(torch.zeros(5, 24), "x", (5,), 24, f, dev) == 24
    assert mb._channels(torch.zeros(1, 40)[:, :24], "x", (1,), 24, f, dev) == 24
    for bad, lead in ((buf[..., ::2], (2, 5)), (buf[:, :4, :20], (2, 4)), (torch.zeros(1, 20).expand(5, 20), (5,)), (torch.zeros(20, 5).t(), (5,))):
        with pytest.raises(ValueError):
            mb._channels(bad, "x", lead, bad.shape[-1], f, dev)
