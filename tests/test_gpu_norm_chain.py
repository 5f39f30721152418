"""GPU: the norm's backward on what its forward returned.  Bounds as in tests/test_gpu_rms_norm.py."""
import pytest
import torch

import layer_forms as lf
import selective_state_space_amd as mb
from gpu_util import require_gpu
from test_gpu_linear_attn import close

pytestmark = pytest.mark.gpu
U, HB = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,D,lead,width", [(9, 200, 0, 264), (5, 33, 3, 40), (1, 64, 8, 80), (4, 1, 0, 3)], ids=str)
def test_backward_of_a_norm_of_rows_that_lie_apart(rows, D, lead, width, dtype):
    """Without a residual r is x itself, here columns of a wider tensor."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(rows, width, generator=g).to(dt).cuda()
    x, w, dy = wide[:, lead:lead + D], 1 + 0.3 * torch.randn(D, generator=g), torch.randn(rows, D, generator=g).to(dt)
    keep = wide.clone()
    y, r, rstd = mb.mb_rms_norm(x, w.cuda())
    assert r is x
    dx, dr, dw = mb.mb_rms_norm_bwd(dy.cuda(), r, rstd, w.cuda())
    want = mb.mb_rms_norm_bwd(dy.cuda(), x.contiguous(), rstd, w.cuda())
    assert all(torch.equal(a, b) for a, b in zip((dx, dr, dw), want)) and torch.equal(wide, keep)
    rr, rw = lf.rms_norm_bwd(dy.double(), x.cpu().double(), rstd.cpu().double(), w.double(), None)
    xh, gw = x.cpu().double() * rstd.cpu().double()[:, None], dy.double() * w.double()
    mag = rstd.cpu().double()[:, None] * (gw.abs() + xh.abs() * (gw * xh).abs().mean(1, keepdim=True))
    close(dx, rr, 100 * U * mag + (HB if dtype == "bf16" else 0) * rr.abs() + 1e-30, "dx")
    close(dw, rw, (100 + rows) * U * (dy.double() * xh).abs().sum(0) + 1e-30, "dw")


def test_other_layouts_are_refused():
    x = torch.randn(6, 4, 8).cuda()
    rstd = torch.ones(6, 4).cuda()
    for r in (torch.randn(6, 4, 16).cuda()[..., ::2], torch.randn(6, 8, 4).cuda().transpose(1, 2), torch.randn(6, 4, 9).cuda()[..., :8]):
        with pytest.raises(ValueError, match="contiguous"):
            mb.mb_rms_norm_bwd(x, r, rstd)
        with pytest.raises(ValueError, match="contiguous"):
            mb.mb_rms_norm(r)
    with pytest.raises(ValueError, match="contiguous"):
        mb.mb_rms_norm_bwd(x[0], torch.randn(8, 4).cuda().t(), rstd[0])
    with pytest.raises(ValueError, match="contiguous"):
        mb.mb_rms_norm_bwd(x[0], torch.randn(1, 8).cuda().expand(4, 8), rstd[0])
