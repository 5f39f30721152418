"""CPU: the float64 definitions that the layer operators are compared with, against automatic
differentiation, central differences and the scans' oracle."""
import numpy as np
import pytest
import torch

import layer_forms as lf

F64 = torch.float64


def _attn_inputs(seed, lens, H, G, Dk, Dv):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=F64)
    T, n = sum(lens), len(lens)
    ld = -torch.rand(H, generator=g, dtype=F64)
    return [rn(T, H, Dk), rn(T, G, Dk), rn(T, G, Dv), rn(n, H, Dk, Dv)], ld, rn(T, H, Dv), rn(n, H, Dk, Dv)


@pytest.mark.parametrize("lens,H,G", [([5], 1, 1), ([3, 0, 4], 4, 2), ([1, 1], 2, 1)])
def test_attention_gradients_are_the_forward_forms(lens, H, G):
    (q, k, v, h0), ld, do, dh = _attn_inputs(1, lens, H, G, 3, 2)
    leaves = [t.clone().requires_grad_() for t in (q, k, v, h0)]
    o, h = lf.attn(*leaves[:3], ld, 0.7, lens, leaves[3])
    ((o * do).sum() + (h * dh).sum()).backward()
    for got, leaf in zip(lf.attn_bwd(q, k, v, ld, 0.7, lens, do, h0, dh), leaves):
        assert torch.allclose(got, leaf.grad, rtol=1e-12, atol=1e-12)


def test_attention_gradients_against_differences():
    lens = [3, 2]
    (q, k, v, h0), ld, do, dh = _attn_inputs(2, lens, 2, 1, 2, 2)

    def loss(q, k, v, h0):
        o, h = lf.attn(q, k, v, ld, 0.5, lens, h0)
        return float((o * do).sum() + (h * dh).sum())

    args, eps = [q, k, v, h0], 1e-5
    for i, got in enumerate(lf.attn_bwd(q, k, v, ld, 0.5, lens, do, h0, dh)):
        for j in range(args[i].numel()):
            hi, lo = args[i].clone(), args[i].clone()
            hi.view(-1)[j] += eps
            lo.view(-1)[j] -= eps
            d = (loss(*args[:i], hi, *args[i + 1:]) - loss(*args[:i], lo, *args[i + 1:])) / (2 * eps)
            assert abs(d - float(got.reshape(-1)[j])) < 1e-8


def test_attention_is_the_ssd_with_a_constant_decay(oracle_mod):
    """The oracle of the Mamba-2 scan with logdecay constant in time and one group per head."""
    (q, k, v, h0), ld, _, _ = _attn_inputs(3, [17], 2, 2, 4, 3)
    o, h = lf.attn(q, k, v, ld, 1.0, [17], h0)
    n = lambda t: np.ascontiguousarray(t.numpy())
    Y, hY = oracle_mod.ssd(n(v)[None], np.tile(n(ld), (1, 17, 1)), n(k)[None], n(q)[None], n(h0))
    assert np.allclose(Y[0], o.numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(hY, h.numpy(), rtol=1e-12, atol=1e-13)


def test_norm_gradient_is_the_forwards():
    g = torch.Generator().manual_seed(4)
    x, res, w, dy, dr_in = (torch.randn(*s, generator=g, dtype=F64) for s in ((4, 7), (4, 7), (7,), (4, 7), (4, 7)))
    leaves = [t.clone().requires_grad_() for t in (x, res, w)]
    y, r, rstd = lf.rms_norm(leaves[0], leaves[2], leaves[1], 1e-5)
    ((y * dy).sum() + (r * dr_in).sum()).backward()
    dr, dw = lf.rms_norm_bwd(dy, r.detach(), rstd.detach(), w, dr_in)
    for got, leaf in zip((dr, dr, dw), leaves):
        assert torch.allclose(got, leaf.grad, rtol=1e-12, atol=1e-12)
    assert torch.allclose(y.detach(), torch.nn.functional.rms_norm(x + res, (7,), w, 1e-5), rtol=1e-12)
