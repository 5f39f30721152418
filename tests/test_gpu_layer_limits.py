"""GPU: the layer operators at the ends of the sizes that they take.  Bounds as in
tests/test_gpu_linear_attn.py and tests/test_gpu_rms_norm.py."""
import pytest
import torch

import layer_forms as lf
import selective_state_space_amd as mb
from gpu_util import require_gpu
from test_gpu_linear_attn import bound, close

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_one_sequence_of_almost_two_to_the_31_tokens():
    """Length and number of segments together pass 2^31.  With a decay of e^-0.25 a token, what lies 300 tokens away weighs
    e^-75 and is left out of the windows' references, which are compared in their middle thirds."""
    T, ld = 2 ** 31 - 5, torch.tensor([-0.25])
    g = torch.Generator(device="cuda").manual_seed(1)

    def fill():
        return torch.empty(1, T, 1, 1, dtype=torch.bfloat16, device="cuda").uniform_(-2.0, 2.0, generator=g)

    q, k, v, do = fill(), fill(), fill(), fill()
    o = torch.full_like(q, float("nan"))
    _, h = mb.mb_linear_attn(q, k, v, ld.cuda(), scale=0.5, o=o)
    grads = mb.mb_linear_attn_bwd(q, k, v, ld.cuda(), do, scale=0.5, dq=torch.full_like(q, float("nan")))
    for t in (o, grads[0]):
        assert not any(bool(torch.isnan(p).any()) for p in t.view(-1).split(2 ** 28)), "tokens that were not written"
    # the first tokens, some of the segments' borders (2^20 tokens each), the last tokens
    for at in (300, 2 ** 20, 2 ** 20 * 777, 2 ** 30, 2 ** 20 * 2047, T - 300):
        w = slice(at - 300, at + 300)
        d = [t[0, w].cpu().double() for t in (q, k, v, do)]
        a = [t.abs() for t in d]
        first, last = 0 if at == 300 else 300, 600 if at == T - 300 else 300      # tokens with all that reaches them
        ro, rh = lf.attn(*d[:3], ld, 0.5, [600])
        Mo, Mh = lf.attn(*a[:3], ld, 0.5, [600])
        tol = bound("bf16", 1, [600], Mo, ro)
        close(o[0, w][first:], ro[first:], tol[first:], "o at %d" % at)
        if at == T - 300:
            close(h, rh, bound("f32", 1, [600], Mh, rh), "h")
        ref, mag = lf.attn_bwd(*d[:3], ld, 0.5, [600], d[3]), lf.attn_bwd(*a[:3], ld, 0.5, [600], a[3])
        for name, got, r, M, part in zip(("dq", "dk", "dv"), grads, ref, mag, (slice(first, 600), slice(0, last), slice(0, last))):
            close(got[0, w][part], r[part], bound("bf16", 5, [600], M, r)[part], name + " at %d" % at)
