"""GPU: the gated linear recurrence with gates far outside where they move, through the C ABI, against the float64 definitions and bounds
of tests/gated_forms.py."""
import pytest
import torch

import gated_forms as gf
import selective_state_space_amd as mb
from gpu_util import require_gpu
from test_gpu_gated_scan import dev, make, offsets, tol, wide
from test_gpu_linear_attn import close

pytestmark = pytest.mark.gpu
NAMES = ("dx", "da_gate", "dx_gate", "ddecay", "da_bias", "dx_bias", "dh0")
INF = float("inf")


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def both(d, lens):
    """(y, h) and the gradients by name, on the GPU and by definition, with the definition's bounds."""
    cu = offsets(lens).cuda()
    kw = dict(a_bias=dev(d["a_bias"]), x_bias=dev(d["x_bias"]), cu_seqlens=cu, h0=d["h0"].cuda())
    ins = [dev(d[k]) for k in ("x", "a_gate", "decay")]
    y, h = mb.mb_gated_scan(*ins, dev(d["x_gate"]), **kw)
    out = dict(zip(NAMES, mb.mb_gated_scan_bwd(*ins, dev(d["dy"]), dev(d["x_gate"]), dh_out=d["dh"].cuda(), **kw)))
    ry, rh, _, ty, th, _ = gf.scan(*wide(d), lens, d["h0"].double())
    ref, bound = gf.scan_bwd(*wide(d), lens, d["dy"].double(), d["h0"].double(), d["dh"].double())
    got, ref, bound = {"y": y, "h": h, **out}, {"y": ry, "h": rh, **ref}, {"y": ty, "h": th, **bound}
    return got, ref, bound


# What a gate far outside gives beside the definition's bounds: an open one's 1 - sigma, and a closed one's sigma, below 2^-120, count as
# any value below 2^-120.  1 - sigma stands in da_gate and dx_gate alone, as a factor.  For a closed decay gate beta is then below
# 2^-58 (decay below 8), so an input adds 2^-58 |x| to a state and G gives 2^-58 G to dx; in da_gate and ddecay b / beta^2 s is below
# 2^-61 |x|.  |x| and |dy| are below 8, a sequence has 170 tokens at most: G, a state and a sum over tokens gather below 2^11 and
# 2^19 of these, all below 2^-38.
FAR = 2.0 ** -38


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("whole", [True, False], ids=["channels", "tokens"])
def test_saturated_gates(whole, dtype):
    """Gates from where e^-v leaves fp32's range on, infinite ones too: values and every gradient, ddecay among them, are those of
    sigma = 1 and 0."""
    lens = [130, 0, 170, 3]
    T, values = sum(lens), [88.0, 90.0, 104.0, 200.0, INF, -88.0, -104.0, -200.0, -INF]
    D = 2 * len(values) + 2
    d = make(71, T, D, dtype, len(lens))
    rows = torch.ones(T, dtype=torch.bool) if whole else torch.rand(T, generator=torch.Generator().manual_seed(72)) < 0.3
    for i, v in enumerate(values):
        d["a_gate"][rows, i] = v
        d["x_gate"][rows, len(values) + i] = v
    d["a_bias"][:len(values)] = 0.0                       # the sums stay on their side of fp32's range
    got, ref, bound = both(d, lens)
    assert bool(d["x"].abs().max() < 8) and bool(d["dy"].abs().max() < 8) and bool(d["decay"].max() < 8)
    for name in ("y", "h") + NAMES:
        wide_type = name in ("h", "ddecay", "da_bias", "dx_bias", "dh0")
        close(got[name], ref[name], tol(bound[name], ref[name], "f32" if wide_type else dtype) + FAR, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_that_their_bias_opens(dtype):
    """The same where a bias of 120 opens the gates of ordinary values."""
    lens, D = [90, 150], 66
    d = make(73, sum(lens), D, dtype, len(lens))
    d["a_bias"][::3], d["x_bias"][1::3] = 120.0, 120.0
    got, ref, bound = both(d, lens)
    for name in ("y", "h") + NAMES:
        wide_type = name in ("h", "ddecay", "da_bias", "dx_bias", "dh0")
        close(got[name], ref[name], tol(bound[name], ref[name], "f32" if wide_type else dtype) + FAR, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_channels_without_memory(dtype):
    """Infinite decay: the outputs do not depend on the decay gate, so that nothing comes to it, its bias and the decay; the rest, and every
    other channel, is as defined."""
    lens, D, none = [70, 0, 200], 18, [0, 7, 17]
    T = sum(lens)
    d = make(75, T, D, dtype, len(lens))
    d["decay"][none] = INF
    d["a_gate"][100:120, 7] = 200.0
    d["a_gate"][30, 17] = INF
    got = both(d, lens)[0]
    d["decay"][none] = 1e30                               # by definition the same values, and bounds that are numbers
    ref, bound = both(d, lens)[1:]
    for name in ("y", "h") + NAMES:
        wide_type = name in ("h", "ddecay", "da_bias", "dx_bias", "dh0")
        close(got[name], ref[name], tol(bound[name], ref[name], "f32" if wide_type else dtype), name)
    for name in ("da_gate", "ddecay", "da_bias"):
        assert bool((got[name][..., none] == 0).all()), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tail", [0, 1, 9, 60, 150])
def test_sums_behind_an_infinite_state(tail, dtype):
    """An infinite last token makes the sums infinite, with the sign that its own share has: the tokens of no sequence behind it, whatever
    they hold, add nothing (not 0 x infinity)."""
    lens, D, c = [60, 40], 34, 5
    T = sum(lens)
    d = make(77, T + tail, D, dtype, len(lens))
    for k in ("x", "a_gate", "x_gate", "dy"):
        d[k][T:] = float("nan")
    d["x"][T - 1, c] = INF
    d["dy"][T - 1, c], d["dh"][1, c] = 1.0, 1.0
    got, _, _ = both(d, lens)
    # of the last token: G = 2, dla = -G a^2 b / beta^2 = -inf; ddecay -dla s, da_gate dla la (1 - s), dx_gate G b (1 - i)
    for name in ("ddecay", "da_bias", "dx_bias"):
        assert float(got[name][c]) == INF, name
    for name in ("dx", "da_gate", "dx_gate"):
        assert bool((got[name][T:] == 0).all()), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sums_of_a_channel_with_an_infinity(dtype):
    """An infinite input in the middle of a sequence: no sum of its channel comes out finite, every other one and the other
    sequences' rows are as without it."""
    lens, D, t, c = [200, 300, 150], 70, 333, 5
    d = make(79, sum(lens), D, dtype, len(lens))
    e = {k: v.clone() for k, v in d.items()}
    e["x"][t, c] = INF
    got, want = both(e, lens)[0], both(d, lens)[0]
    for name in NAMES:
        g, w = got[name].cpu().clone(), want[name].cpu()
        if name in ("ddecay", "da_bias", "dx_bias"):
            assert not bool(torch.isfinite(g[c])), name
            g[c] = w[c]
        elif name == "dh0":
            g[1, c] = w[1, c]
        else:
            g[200:500, c] = w[200:500, c]
        assert torch.equal(g, w), name
