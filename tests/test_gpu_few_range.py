"""Values of very different size within a row of x or of H, where the smallest digits
of the 4-bit layer's x and H decide the output, against the 64-bit form of few_check.

x: one element of every row is 2^28 units, and its weights are 0, so that a unit's sum
is that of the others, whole numbers of up to 255 units 2^s (s below): with the
largest magnitude in [2^29, 2^30) the layer's unit is half of theirs and x enters
exactly.  The output is then that of the row without the large element, to the bound
of that row.  (A layer that kept 23 bits of the row would have a unit of 2^7.)

H: units 5, 37, 69, .. are some 2^20 times the others and their rows of w2 are 0.  The
output is that of the layer without those units, whose bound gains what the rounding
to 2^-30 of the largest |g H| adds, g 2^-30 max |H| sum |w2|.  Two units of the others
reach a column of the output, so that this stays small: 2^-9 of a typical output.
"""

import pytest
import torch

import few_check as F
import sparse_mixture_experts_22_b200 as M
from test_gpu_few import make_layer, run
from sparse_mixture_experts_22_b200 import inputs as I
from sparse_mixture_experts_22_b200.workloads import Workload

pytestmark = pytest.mark.gpu

# every expert serves every token: 1 to 8 tiles of the tokens' digits, the last one
# full and half full
TOKENS = [1, 2, 3, 4, 5, 6, 7, 8, 9, 12, 15, 16]


def values(inp, group):
    """The weights that the layer stands for, in 64 bits."""
    return [F.quantize(inp[n].transpose(1, 2), group)[2].transpose(1, 2) if group
            else inp[n].double() for n in ("w1", "w3", "w2")]


@pytest.mark.parametrize("shift", [0, 8, 16])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("T", TOKENS)
def test_a_large_element_of_x(T, group, shift):
    wl = Workload("f_range", T=T, d=256, h=256, E=2, k=2)
    inp = dict(I.layer_inputs(wl))
    gen = torch.Generator().manual_seed(100 * T + group + shift)
    units = torch.randint(-255, 256, (T, wl.d), generator=gen).double() * 2.0 ** shift
    at = torch.randint(0, wl.d, (1,), generator=gen).item()
    units[:, at] = 0
    x0 = (units * 2.0 ** (-8 - shift)).to(torch.bfloat16)
    assert torch.equal(x0.double(), units * 2.0 ** (-8 - shift))
    for n in ("w1", "w3"):
        inp[n] = inp[n].clone()
        inp[n][:, at, :] = 0
    inp["Wr"] = inp["Wr"].clone()
    inp["Wr"][at] = 0
    w = values(inp, group)
    ref = F.layer(x0, inp["Wr"], inp["bias"], wl.k, *w, None, None, group > 0)
    assert float(ref["out"].abs().max()) > 0
    x = x0.clone()
    x[:, at] = torch.tensor([1.0, -1.0]).repeat(T)[:T].to(torch.bfloat16) * 2.0 ** (20 - shift)
    inp["x"] = x
    layer, g = make_layer(wl, inp, group)
    F.check(run(layer, g["x"]), ref)


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("T,h,E", [(t, 128, 2) for t in TOKENS] + [(2, 4096, 4), (7, 2048, 8)])
def test_large_elements_of_h(T, h, E, group):
    wl = Workload("f_range_h", T=T, d=256, h=h, E=E, k=min(E, 4))
    inp = dict(I.layer_inputs(wl))
    gen = torch.Generator().manual_seed(T + h + group)
    large = torch.arange(5, h, 32)
    small = torch.tensor([j for j in range(h) if j % 32 != 5])
    for n in ("w1", "w3"):
        inp[n] = inp[n].clone()
        inp[n][:, :, large] *= 2.0 ** 10
    w2 = torch.zeros(E, h, wl.d)
    for e in range(E):
        for _ in range(2):
            rows = small[torch.randint(0, len(small), (wl.d,), generator=gen)]
            w2[e, rows, torch.arange(wl.d)] = torch.randn(wl.d, generator=gen)
    inp["w2"] = w2.bfloat16()
    w = values(inp, group)
    # the same layer without the large units
    wo = [v.clone() for v in w]
    for v in wo[:2]:
        v[:, :, large] = 0
    ref = F.layer(inp["x"], inp["Wr"], inp["bias"], wl.k, *wo, None, None, group > 0)
    if group:
        x = inp["x"].double()
        for t in range(T):
            for j in range(wl.k):
                e = int(ref["idx"][t, j])
                a, u = x[t] @ w[0][e], x[t] @ w[1][e]
                most = (a * torch.sigmoid(a) * u).abs().max()
                ref["bound"][t] += ref["gate"][t, j] * 2.0 ** -30 * most * w[2][e].abs().sum(0)
    layer, g = make_layer(wl, inp, group)
    F.check(run(layer, g["x"]), ref)
