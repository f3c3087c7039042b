"""A FewLayer keeps to the config it was made with, and refuses what it lacks."""

import pytest
import torch

import few_check as F
import sparse_mixture_experts_22_b200 as M
from test_gpu_few import device_weights, made

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [0, 64])
def test_a_config_changed_later(group):
    """The caller's struct goes on to another use: batch sizes seen and not seen before
    stay what they were, and no larger batch is taken."""
    wl, inp, ref = made("capped", group)
    cfg, g, W = device_weights(wl, inp)
    W = list(M.quantize_weights(cfg, *W, group)) if group else W
    layer = M.FewLayer(cfg, g["Wr"], g["bias"], *W, group=group or None)
    few = {t: {n: v.clone() for n, v in layer(g["x"][:t].contiguous()).items()} for t in (3, wl.T)}
    seen = M.FewLayer(cfg, g["Wr"], g["bias"], *W, group=group or None)
    seen(g["x"])
    cfg.T, cfg.cf_num, cfg.cf_den, cfg.has_bias = 16, 0, 0, 0
    F.check(seen(g["x"]), ref)
    fresh = seen(g["x"][:3].contiguous())
    for n, v in few[3].items():
        assert torch.equal(fresh[n], v), n
    with pytest.raises(ValueError):
        seen(torch.zeros((wl.T + 1, wl.d), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("missing", ["bias", "W13", "W2p", "W13s", "W2s"])
def test_missing_inputs(missing):
    wl, inp, _ = made("shared")
    cfg, g, W = device_weights(wl, inp)
    cfg.has_bias = 1
    args = dict(zip(("bias", "W13", "W2p", "W13s", "W2s"), (torch.zeros(wl.E, device="cuda"), *W)))
    M.FewLayer(cfg, g["Wr"], **args)
    args[missing] = None
    with pytest.raises(ValueError):
        M.FewLayer(cfg, g["Wr"], **args)
