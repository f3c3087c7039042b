"""Host-side checks of the few-token layer and the 4-bit weights: sizes,
refusals before any launch, and the plain 64-bit form against the fp64 oracle."""

import ctypes

import numpy as np
import pytest
import torch

import few_check as F
import oracle as O
import sparse_mixture_experts_22_b200 as M
from sparse_mixture_experts_22_b200 import binding as B
from sparse_mixture_experts_22_b200 import build as build_mod
from sparse_mixture_experts_22_b200 import inputs as I
from sparse_mixture_experts_22_b200.workloads import WORKLOADS, Workload


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


def test_sizes():
    # 4.5 bits a weight at a group of 32, 4.25 at 64, 4.125 at 128
    for group, bits in ((32, 4.5), (64, 4.25), (128, 4.125)):
        cfg = M.make_config(1, 640, 896, 5, 2, n_shared=2, h_shared=128)
        a, b = M.moe_q4_size(cfg, 0, group)
        assert a == 5 * 2 * 896 * 640 * bits / 8 and b == 5 * 640 * 896 * bits / 8
        a, b = M.moe_q4_size(cfg, 1, group)
        assert a == 2 * 256 * 640 * bits / 8 and b == 640 * 256 * bits / 8
    assert M.moe_few_workspace_size(M.make_config(0, 128, 128, 4, 2)) >= 256
    sizes = [M.moe_few_workspace_size(M.make_config(t, 5120, 1536, 160, 6, 2, 1536))
             for t in range(1, M.MOE_FEW_MAX_T + 1)]
    assert all(0 < s < 256 << 20 for s in sizes)


@pytest.mark.parametrize("kw,code", [
    (dict(T=17, d=128, h=128, E=4, k=2), 2),
    (dict(T=4, d=100, h=128, E=4, k=2), 2),
    (dict(T=4, d=128, h=128, E=4, k=2, dtype="f32"), 3),
    (dict(T=4, d=128, h=128, E=4, k=2, cf=(5, 4), overflow="reroute"), 8),
    (dict(T=4, d=128, h=128, E=4, k=2, train=True), 8),
])
def test_configs_the_few_layer_refuses(kw, code):
    with pytest.raises(B.MoEError) as e:
        M.moe_few_workspace_size(M.make_config(**kw))
    assert e.value.code == code


def _call(name, cfg, *args):
    rc = getattr(B.load(), name)(ctypes.byref(cfg), *args)
    return rc, B.load().moe_last_error().decode()


def _ptrs(n, base=1 << 20):
    return [ctypes.c_void_p(base + 4096 * i) for i in range(n)]


def test_refusals_before_any_launch():
    cfg = M.make_config(4, 128, 128, 4, 2, n_shared=1, h_shared=128, has_bias=True)
    size = M.moe_few_workspace_size(cfg)
    names = ["x", "Wr", "bias", "W13", "W2p", "W13s", "W2s", "out", "topk_idx", "topk_gate",
             "routed", "kept", "stats"]
    base = _ptrs(len(names)) + [ctypes.c_void_p(1 << 16), size, None]
    ws = len(names)

    def run(i, value):
        a = list(base)
        a[i] = value
        return _call("moe_forward_few", cfg, *a)

    for i, n in enumerate(names):
        if n != "stats":
            rc, msg = run(i, None)
            assert rc == 1 and n in msg, (n, rc, msg)
        rc, msg = run(i, ctypes.c_void_p((1 << 20) + 8))
        assert rc == 4 and n in msg, (n, rc, msg)
    assert run(ws, None)[0] == 1
    assert run(ws, ctypes.c_void_p((1 << 16) + 128))[0] == 4
    assert run(ws + 1, size - 1)[0] == 5
    assert run(names.index("out"), base[0])[0] == 1  # out aliases x
    for group in (0, -32, 16, 96, 256):
        assert _call("moe_forward_few_q4", cfg, group, *base)[0] == 1
        with pytest.raises(B.MoEError) as e:
            M.moe_q4_size(cfg, 0, group)
        assert e.value.code == 1


def test_refusals_of_the_4_bit_calls():
    cfg = M.make_config(4, 128, 128, 4, 2)
    for name in ("moe_q4_quantize", "moe_q4_dequantize"):
        for i in range(4):
            a = _ptrs(4)
            a[i] = None
            assert _call(name, cfg, 0, 64, *a, None)[0] == 1
            a[i] = ctypes.c_void_p((1 << 20) + 8)
            assert _call(name, cfg, 0, 64, *a, None)[0] == 4
        assert _call(name, cfg, 0, 48, *_ptrs(4), None)[0] == 1
        assert _call(name, cfg, 1, 64, *_ptrs(4), None)[0] == 1   # no shared experts
        assert _call(name, cfg, 2, 64, *_ptrs(4), None)[0] == 1
        f32 = M.make_config(4, 128, 128, 4, 2, dtype="f32")
        assert _call(name, f32, 0, 64, *_ptrs(4), None)[0] == 3


def test_tensors_the_binding_refuses():
    cfg = M.make_config(2, 128, 128, 3, 2)
    W13, W2p = torch.zeros(3, 256, 128).bfloat16(), torch.zeros(3, 128, 128).bfloat16()
    with pytest.raises(ValueError):
        M.quantize_weights(cfg, W13, W2p)                       # not on a GPU
    with pytest.raises(ValueError):
        M.FewLayer(cfg, torch.zeros(128, 3), None, W13, W2p)


@pytest.mark.parametrize("wl", [
    Workload("c", T=9, d=128, h=128, E=5, k=2, n_shared=2, h_shared=128, cf=(5, 4), zipf_s=0.7),
    WORKLOADS["tiny"].scaled(T=5),
], ids=["capped_shared", "tiny"])
def test_plain_form_equals_the_oracle(wl):
    inp = I.layer_inputs(wl)
    shared = (inp["w1s"], inp["w3s"], inp["w2s"]) if wl.n_shared else None
    ref = F.layer(inp["x"], inp["Wr"], inp["bias"], wl.k, inp["w1"], inp["w3"], inp["w2"], shared,
                  wl.cf)
    r = O.forward(O.cfg_of(wl), inp)
    assert np.array_equal(ref["idx"].numpy(), r["idx"])
    assert ref["routed"] == r["routed"].tolist() and ref["kept"] == r["kept"].tolist()
    assert np.abs(ref["out"].numpy() - r["out"]).max() <= 1e-12 * np.abs(r["out"]).max() + 1e-12
    assert np.abs(ref["gate"].numpy() - r["gate"]).max() <= 1e-14


def test_plain_quantisation():
    # a / 7 = 0.5 exactly: halves go to the even code, the largest weight to 7
    w = torch.tensor([[3.5, -3.5, 0.25, 0.75, -0.25, 1.2, 0.0, 2.9] + [0.0] * 24]).bfloat16()
    q, s, v = F.quantize(w, 32)
    assert float(s) == 0.5
    assert q[0, :8].tolist() == [7, -7, 0, 2, 0, 2, 0, 6]
    z = F.quantize(torch.zeros(1, 64), 64)
    assert float(z[1]) == 0 and not z[0].any()


@pytest.mark.parametrize("name", ["moe_q4_quantize", "moe_q4_dequantize"])
def test_4_bit_calls_refuse_overlapping_sets(name):
    cfg = M.make_config(4, 128, 128, 4, 2)
    w = [1 << 30, 1 << 31]
    sizes = [2 * 4 * 128 * 128 * 2, 4 * 128 * 128 * 2]
    q13, q2 = M.moe_q4_size(cfg, 0, 64)
    for i in range(2):
        for j, q in enumerate((q13, q2)):
            for at in (w[i], w[i] + sizes[i] - 16, w[i] - q + 16):  # each end, by 16 bytes
                qs = [1 << 32, 1 << 33]
                qs[j] = at
                order = w + qs if name == "moe_q4_quantize" else qs + w
                rc, msg = _call(name, cfg, 0, 64, *(ctypes.c_void_p(p) for p in order), None)
                assert rc == 1 and "overlap" in msg, (i, j, rc, msg)
