"""CPU: what the layer operators refuse, on the host and before anything is enqueued (no pointer
here is ever dereferenced)."""
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


def attn(lib, q=M, k=2 * M, v=3 * M, ld=4 * M, cu=0, h0=0, has=0, slots=0, o=5 * M, h=6 * M, n=2, T=200, H=4, G=2, Dk=64, Dv=64,
         ns=0, qs=256, ks=128, vs=128, dt=F32, ws=7 * M, nws=M):
    return lib.mb_linear_attn(p(q), p(k), p(v), p(ld), p(cu), p(h0), p(has), p(slots), p(o), p(h), n, T, H, G, Dk, Dv, ns, qs, ks, vs,
                              1.0, dt, p(ws), nws, None)


def test_linear_attn(lib):
    for dt in (2, 7, -1):
        assert attn(lib, dt=dt) == E_DTYPE
    for kw in (dict(n=-1), dict(T=-1), dict(H=0), dict(G=0), dict(G=3), dict(Dk=0), dict(Dk=129), dict(Dv=0), dict(Dv=129), dict(T=201),
               dict(qs=255), dict(ks=127), dict(vs=1), dict(T=1 << 31), dict(n=(1 << 20) + 1), dict(H=4097, G=4097),
               dict(qs=1 << 22), dict(slots=8 * M, ns=1 << 31), dict(ns=3), dict(slots=8 * M, ns=0), dict(slots=8 * M, ns=-1)):
        assert attn(lib, **kw) == E_SHAPE, kw
    for kw in (dict(q=0), dict(k=0), dict(v=0), dict(o=0), dict(ld=0)):
        assert attn(lib, **kw) == E_NULL, kw
    for kw in (dict(q=M + 2), dict(o=5 * M + 1), dict(ld=4 * M + 2), dict(cu=8 * M + 2), dict(h=6 * M + 1), dict(q=M + 1, dt=BF16)):
        assert attn(lib, **kw) == E_ALIGN, kw
    for kw in (dict(o=M + 64), dict(h=2 * M), dict(h0=6 * M + 4), dict(o=6 * M), dict(o=4 * M)):
        assert attn(lib, **kw) == E_ALIAS, kw
    big = dict(T=4000, n=1, cu=8 * M)
    need = mb.mb_workspace_size(mb.MB_OP_LINEAR_ATTN, 1, 4000, 4, 64, 2, 64)
    assert need > 0
    assert attn(lib, **big, nws=need - 1) == E_WS
    assert attn(lib, **big, ws=0, nws=0) == E_WS
    assert attn(lib, **big, ws=7 * M + 16) == E_WS
    assert attn(lib, **big, ws=6 * M) == E_ALIAS
    assert attn(lib, **big, ws=M) == E_ALIAS
    assert attn(lib, n=0) == OK
    assert mb.mb_workspace_size(mb.MB_OP_LINEAR_ATTN, 1, 4000, 4, 64, 2, 200) == 0


def step(lib, q=M, k=2 * M, v=3 * M, ld=4 * M, slots=0, hi=6 * M, ho=6 * M, o=5 * M, n=2, H=4, G=2, Dk=64, Dv=64, ns=0, qs=256, ks=128,
         vs=128, dt=F32):
    return lib.mb_linear_attn_step(p(q), p(k), p(v), p(ld), p(slots), p(hi), p(ho), p(o), n, H, G, Dk, Dv, ns, qs, ks, vs, 1.0, dt, None)


def test_linear_attn_step(lib):
    assert step(lib, dt=2) == E_DTYPE
    for kw in (dict(n=-1), dict(G=3), dict(Dk=129), dict(Dv=0), dict(qs=255), dict(ns=1), dict(slots=8 * M)):
        assert step(lib, **kw) == E_SHAPE, kw
    for kw in (dict(q=0), dict(ho=0), dict(o=0), dict(ld=0)):
        assert step(lib, **kw) == E_NULL, kw
    assert step(lib, ho=6 * M + 64) == E_ALIAS
    assert step(lib, o=M) == E_ALIAS
    assert step(lib, o=6 * M) == E_ALIAS
    assert step(lib, hi=6 * M + 2) == E_ALIGN
    assert step(lib, n=0) == OK


def bwd(lib, q=M, k=2 * M, v=3 * M, ld=4 * M, cu=0, h0=0, do=5 * M, dh=0, dq=6 * M, dk=7 * M, dv=8 * M, dh0=9 * M, n=1, T=200, H=4, G=2,
        Dk=64, Dv=64, qs=256, ks=128, vs=128, dt=F32, ws=10 * M, nws=M):
    return lib.mb_linear_attn_bwd(p(q), p(k), p(v), p(ld), p(cu), p(h0), p(do), p(dh), p(dq), p(dk), p(dv), p(dh0), n, T, H, G, Dk, Dv,
                                  qs, ks, vs, 1.0, dt, p(ws), nws, None)


def test_linear_attn_bwd(lib):
    assert bwd(lib, dt=2) == E_DTYPE
    for kw in (dict(n=-1), dict(G=3), dict(Dk=129), dict(Dv=0), dict(qs=255), dict(n=3)):
        assert bwd(lib, **kw) == E_SHAPE, kw
    for kw in (dict(q=0), dict(do=0), dict(dq=0), dict(dk=0), dict(dv=0), dict(ld=0)):
        assert bwd(lib, **kw) == E_NULL, kw
    for kw in (dict(dq=M), dict(dk=6 * M), dict(dv=5 * M), dict(dh0=8 * M), dict(dh=9 * M), dict(ws=6 * M), dict(ws=5 * M)):
        assert bwd(lib, **kw) == E_ALIAS, kw
    need = mb.mb_workspace_size(mb.MB_OP_LINEAR_ATTN_BWD, 1, 200, 4, 64, 2, 64)
    assert need > 0                                       # shared keys: the heads' gradients before they are added up
    assert bwd(lib, nws=need - 1) == E_WS
    assert bwd(lib, do=5 * M + 1) == E_ALIGN
    assert bwd(lib, n=0) == E_SHAPE                       # tokens, but no sequence to hold them
    assert bwd(lib, n=0, T=0) == OK


def norm(lib, x=M, res=2 * M, w=3 * M, y=4 * M, ro=5 * M, rs=6 * M, rows=4, D=64, xs=64, eps=1e-5, dt=BF16, rdt=F32):
    return lib.mb_rms_norm(p(x), p(res), p(w), p(y), p(ro), p(rs), rows, D, xs, eps, dt, rdt, None)


def norm8(lib, sc=7 * M, group=32, y=4 * M, rows=4, D=64):
    return lib.mb_rms_norm_fp8(p(M), None, None, p(y), p(sc), None, None, rows, D, D, group, 1e-5, BF16, F32, None)


def test_rms_norm(lib):
    for kw in (dict(dt=2), dict(rdt=3), dict(dt=F32, rdt=BF16)):
        assert norm(lib, **kw) == E_DTYPE, kw
    for kw in (dict(rows=-1), dict(D=0), dict(D=16385, xs=16385), dict(xs=63), dict(xs=1 << 31), dict(eps=-1.0), dict(eps=INF), dict(eps=float("nan")),
               dict(rows=(1 << 30) + 1)):
        assert norm(lib, **kw) == E_SHAPE, kw
    for kw in (dict(x=0), dict(y=0)):
        assert norm(lib, **kw) == E_NULL, kw
    for kw in (dict(x=M + 1), dict(res=2 * M + 2), dict(w=3 * M + 2), dict(rs=6 * M + 1)):
        assert norm(lib, **kw) == E_ALIGN, kw
    for kw in (dict(y=M), dict(y=2 * M), dict(ro=2 * M + 4), dict(ro=M), dict(rs=4 * M), dict(ro=4 * M), dict(y=3 * M)):
        assert norm(lib, **kw) == E_ALIAS, kw
    assert norm(lib, rows=0) == OK
    for g in (16, 48, 256, -1):
        assert norm8(lib, group=g) == E_SHAPE
    assert norm8(lib, sc=0) == E_NULL
    assert norm8(lib, sc=4 * M) == E_ALIAS
    assert norm8(lib, y=M) == E_ALIAS
    assert norm8(lib, rows=0) == OK


def nbwd(lib, dy=M, r=2 * M, rs=3 * M, w=4 * M, din=0, dx=5 * M, dr=6 * M, dw=7 * M, rows=5000, D=64, dt=BF16, rdt=F32, ws=8 * M, nws=M):
    return lib.mb_rms_norm_bwd(p(dy), p(r), p(rs), p(w), p(din), p(dx), p(dr), p(dw), rows, D, dt, rdt, p(ws), nws, None)


def test_rms_norm_bwd(lib):
    for kw in (dict(dt=2), dict(dt=F32, rdt=BF16)):
        assert nbwd(lib, **kw) == E_DTYPE
    for kw in (dict(rows=-1), dict(D=0), dict(D=16385)):
        assert nbwd(lib, **kw) == E_SHAPE
    for kw in (dict(dy=0), dict(r=0), dict(rs=0), dict(dx=0, dr=0, dw=0)):
        assert nbwd(lib, **kw) == E_NULL, kw
    for kw in (dict(dx=M), dict(dr=2 * M), dict(dw=4 * M), dict(din=6 * M + 4), dict(dr=5 * M), dict(ws=5 * M), dict(ws=M)):
        assert nbwd(lib, **kw) == E_ALIAS, kw
    need = mb.mb_workspace_size(mb.MB_OP_RMS_NORM_BWD, 5000, 1, 64, 1, 1, 1)
    assert need > 0 and nbwd(lib, nws=need - 1) == E_WS and nbwd(lib, ws=0) == E_WS and nbwd(lib, ws=8 * M + 8) == E_WS
    assert mb.mb_workspace_size(mb.MB_OP_RMS_NORM_BWD, 1, 1, 64, 1, 1, 1) == 0
    assert nbwd(lib, r=2 * M + 2) == E_ALIGN


def clip(lib, g=(M, 2 * M), o=None, sizes=(100, 200), n=None, mx=1.0, eps=1e-6, norm=3 * M, dt=F32, ws=4 * M, nws=M):
    k = len(g)
    arr = lambda v: ctypes.cast((ctypes.c_void_p * k)(*v), ctypes.c_void_p)
    return lib.mb_grad_norm_clip(arr(g), None if o is None else arr(o), ctypes.cast((ctypes.c_int64 * k)(*sizes), ctypes.c_void_p),
                                 k if n is None else n, mx, eps, p(norm), dt, p(ws), nws, None)


def test_grad_norm_clip(lib):
    assert clip(lib, dt=2) == E_DTYPE
    for kw in (dict(n=-1), dict(n=65537), dict(sizes=(1, -1)), dict(mx=-1.0), dict(mx=float("nan")), dict(eps=-1.0), dict(eps=INF)):
        assert clip(lib, **kw) == E_SHAPE, kw
    for kw in (dict(norm=0), dict(g=(M, 0)), dict(o=(M, 0))):
        assert clip(lib, **kw) == E_NULL, kw
    for kw in (dict(g=(M + 2, 2 * M)), dict(norm=3 * M + 2), dict(o=(5 * M + 1, 6 * M))):
        assert clip(lib, **kw) == E_ALIGN, kw
    for kw in (dict(o=(M + 4, 6 * M)), dict(norm=M + 8), dict(g=(M, 4 * M)), dict(ws=3 * M)):
        assert clip(lib, **kw) == E_ALIAS, kw
    need = mb.mb_workspace_size(mb.MB_OP_GRAD_NORM_CLIP, 2, 1, 1, 1, 1, 1)
    for kw in (dict(nws=need - 1), dict(ws=0), dict(ws=4 * M + 64)):
        assert clip(lib, **kw) == E_WS, kw


def test_grad_norm_clip_of_tensors_that_overlap(lib):
    """Every pair in which one is written."""
    K = 1024
    assert clip(lib, g=(M, M), sizes=(K, K)) == E_ALIAS                                # the same tensor twice
    assert clip(lib, g=(M, M + 4 * K - 4), sizes=(K, K)) == E_ALIAS
    assert clip(lib, g=(M + 4 * K - 4, M), sizes=(K, K)) == E_ALIAS                    # in either order
    assert clip(lib, g=(M, 6 * M), o=(7 * M, M), sizes=(K, K)) == E_ALIAS              # written on another one's gradient
    assert clip(lib, g=(M, 2 * M), o=(7 * M, 7 * M + 8), sizes=(K, K)) == E_ALIAS      # two outputs
    assert clip(lib, g=tuple(M + 4 * K * i for i in range(400)) + (M,), sizes=(K,) * 401) == E_ALIAS



def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 8)
    q = torch.zeros(1, 3, 2, 8)
    for call in (lambda: mb.mb_rms_norm(x), lambda: mb.mb_rms_norm_fp8(x), lambda: mb.mb_rms_norm_bwd(x, x, x[:, 0]),
                 lambda: mb.mb_grad_norm_clip([x], 1.0), lambda: mb.mb_linear_attn(q, q, q, x[0, :2]),
                 lambda: mb.mb_linear_attn_step(q[0], q[0], q[0], x[0, :2], q), lambda: mb.mb_linear_attn_bwd(q, q, q, x[0, :2], q)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="at least one"):
        mb.mb_grad_norm_clip([], 1.0)


def test_binding_token_strides():
    """The stride of a token in views of a fused projection, and the layouts that have none."""
    dev, f = torch.device("cpu"), torch.float32
    wide = torch.zeros(2, 5, 40)
    q = wide[..., 8:32].unflatten(-1, (3, 8))
    assert mb._tokens(q, "q", (2, 5), 3, 8, f, dev) == 40
    assert mb._tokens(wide[0, :, :24].unflatten(-1, (3, 8)), "q", (5,), 3, 8, f, dev) == 40
    assert mb._tokens(torch.zeros(2, 5, 3, 8), "q", (2, 5), 3, 8, f, dev) == 24
    assert mb._tokens(torch.zeros(2, 5, 1, 8)[:, :1], "q", (2, 1), 1, 8, f, dev) == 40
    for bad, lead, h, w in ((torch.zeros(2, 3, 5, 8).transpose(1, 2), (2, 5), 3, 8), (wide[:, :4, :24].unflatten(-1, (3, 8)), (2, 4), 3, 8),
                            (torch.zeros(1, 1, 3, 8).expand(2, 5, 3, 8), (2, 5), 3, 8), (torch.zeros(5, 3, 16)[..., ::2], (5,), 3, 8)):
        with pytest.raises(ValueError):
            mb._tokens(bad, "q", lead, h, w, f, dev)
