"""GPU: linear attention in bf16 rounds nothing but its outputs to bf16.

Scores and the state's copy reach the matrix products as two bf16 pieces: the first is off by at most h = 2^-8 of a value, the
second, of what the first leaves, by h of that: h^2 = 2^-16 of every term. So beside the fp32 bound (see
tests/test_gpu_linear_attn.py) 2^-16 of the magnitudes M, and h of the result itself for its own rounding.  Inputs have both
signs: many results are far smaller than M, and a single rounding of the operands would show in them."""
import pytest
import torch

import layer_forms as lf
import selective_state_space_amd as mb
from gpu_util import require_gpu
from test_gpu_linear_attn import HB, _id, bound, close, decays, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def tight(Dk, lens, M, ref):
    return bound("f32", Dk, lens, M, ref) + HB * HB * M + HB * ref.abs()


CASES = [  # lens, H, G, Dk, Dv, decay
    ([65], 1, 1, 16, 16, "mixed"), ([300], 2, 2, 64, 64, "none"), ([5, 0, 700, 64], 4, 2, 128, 64, "mixed"), ([1100, 3], 2, 1, 72, 100, "mixed"),
    ([900, 200], 2, 2, 128, 128, "none"), ([1500], 2, 2, 64, 128, "mixed"), ([400], 2, 1, 17, 33, "mixed"), ([300], 2, 2, 128, 20, "strong")]


@pytest.mark.parametrize("case", CASES, ids=_id)
def test_outputs_and_gradients(case):
    lens, H, G, Dk, Dv, kind = case
    T, n, ld, scale = sum(lens), len(lens), decays(H, kind), 0.3
    d = inputs(101, T, H, G, Dk, Dv, "bf16", n, with_do=True)
    cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32).cuda()
    c = {x: t.cuda() for x, t in d.items()}
    D = {x: t.double() for x, t in d.items()}
    A = {x: t.abs() for x, t in D.items()}
    o, _ = mb.mb_linear_attn(c["q"], c["k"], c["v"], ld.cuda(), scale=scale, cu_seqlens=cu, h0=c["h0"])
    ro, _ = lf.attn(D["q"], D["k"], D["v"], ld, scale, lens, D["h0"])
    Mo, _ = lf.attn(A["q"], A["k"], A["v"], ld, scale, lens, A["h0"])
    close(o, ro, tight(Dk, lens, Mo, ro), "o")
    out = mb.mb_linear_attn_bwd(c["q"], c["k"], c["v"], ld.cuda(), c["do"], scale=scale, cu_seqlens=cu, h0=c["h0"], dh_out=c["dh"])
    ref = lf.attn_bwd(D["q"], D["k"], D["v"], ld, scale, lens, D["do"], D["h0"], D["dh"])
    mag = lf.attn_bwd(A["q"], A["k"], A["v"], ld, scale, lens, A["do"], A["h0"], A["dh"])
    for name, got, r, M in zip(("dq", "dk", "dv"), out, ref, mag):
        close(got, r, tight(max(Dk, Dv) + 4 * (H // G), lens, M, r), name)


@pytest.mark.parametrize("widths", [(64, 64), (128, 64), (64, 128)], ids=str)
def test_tokens_in_front_of_an_infinity(widths):
    """The products that leave out later tokens one by one keep both pieces."""
    (Dk, Dv), H, L = widths, 2, 200
    ld = decays(H)
    d = inputs(102, L, H, H, Dk, Dv, "bf16", 1, with_do=True)
    D = {x: t.double() for x, t in d.items()}
    A = {x: t.abs() for x, t in D.items()}
    ro, _ = lf.attn(D["q"], D["k"], D["v"], ld, 0.3, [L], D["h0"])
    Mo, _ = lf.attn(A["q"], A["k"], A["v"], ld, 0.3, [L], A["h0"])
    d["v"][150, :, 7] = float("inf")
    cu = torch.tensor([0, L], dtype=torch.int32).cuda()
    o, _ = mb.mb_linear_attn(*(d[x].cuda() for x in "qkv"), ld.cuda(), scale=0.3, cu_seqlens=cu, h0=d["h0"].cuda())
    close(o[:150], ro[:150], tight(Dk, [L], Mo, ro)[:150], "o")
    d["v"][150, :, 7] = 1.0
    d["do"][150, :, 7] = float("inf")
    D["v"][150, :, 7] = A["v"][150, :, 7] = 1.0
    dq, dk, dv, _ = mb.mb_linear_attn_bwd(*(d[x].cuda() for x in "qkv"), ld.cuda(), d["do"].cuda(), scale=0.3, cu_seqlens=cu, h0=d["h0"].cuda())
    ref = lf.attn_bwd(D["q"], D["k"], D["v"], ld, 0.3, [L], D["do"], D["h0"])
    mag = lf.attn_bwd(A["q"], A["k"], A["v"], ld, 0.3, [L], A["do"], A["h0"])
    close(dk[151:], ref[1][151:], tight(max(Dk, Dv) + 4, [L], mag[1], ref[1])[151:], "dk")
    close(dv[151:], ref[2][151:], tight(max(Dk, Dv) + 4, [L], mag[2], ref[2])[151:], "dv")
