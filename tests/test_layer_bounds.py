"""CPU: the bounds of the long linear attention tests are narrow enough: a token that is left out of one result, or a
segment that is left out of the state entering the next, lies outside them."""
import pytest
import torch

import layer_forms as lf
from test_gpu_linear_attn import bound
from test_gpu_linear_attn_long import positive

LD, D = torch.tensor([-0.05, -0.0005]), 64


def _inputs(T):
    d = positive(5, T, 2, 2, D, D, "bf16", 1)
    return [d[x].double() for x in ("q", "k", "v", "do", "h0", "dh")]


@pytest.mark.parametrize("t", [0, 37, 63, 64, 200, 298, 299])
def test_a_token_left_out_is_seen(t):
    T = 300
    q, k, v, do, h0, dh = _inputs(T)
    ro, rh = lf.attn(q, k, v, LD, D ** -0.5, [T], h0)
    ref = lf.attn_bwd(q, k, v, LD, D ** -0.5, [T], do, h0, dh)
    without = lambda x: torch.cat([x[:t], torch.zeros_like(x[:1]), x[t + 1:]])
    o, _ = lf.attn(q, without(k), v, LD, D ** -0.5, [T], h0)
    assert bool(((o - ro).abs() > bound("bf16", D, [T], ro, ro)).any())
    dq = lf.attn_bwd(q, without(k), v, LD, D ** -0.5, [T], do, h0, dh)[0]
    dk, dv = lf.attn_bwd(q, k, v, LD, D ** -0.5, [T], without(do), h0, dh)[1:3]
    for got, r in ((dq, ref[0]), (dk, ref[1]), (dv, ref[2])):
        assert bool(((got - r).abs() > bound("bf16", D, [T], r, r)).any())


def test_a_segment_left_out_is_seen():
    T, a, b = 1280, 512, 768
    q, k, v, _, h0, _ = _inputs(T)
    h0 = 0.01 * h0
    ro, _ = lf.attn(q, k, v, LD, D ** -0.5, [T], h0)
    k2 = k.clone()
    k2[a:b] = 0
    o, _ = lf.attn(q, k2, v, LD, D ** -0.5, [T], h0)
    # in the segment behind the next one: only the slow head holds it
    assert bool(((o - ro).abs() > bound("bf16", D, [T], ro, ro))[b + 256:, 1].any())
