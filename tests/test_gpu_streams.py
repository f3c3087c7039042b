"""Calls of the layer that allocate their results, on a given stream: no call writes
memory that another stream still reads, and no memory is handed out again under a call.
A stream is held up by a kernel that only waits some 20 ms."""

import pytest
import torch

import sparse_mixture_experts_22_b200 as M
from sparse_mixture_experts_22_b200 import inputs as I
from sparse_mixture_experts_22_b200.workloads import Workload

pytestmark = pytest.mark.gpu

CYCLES = 40_000_000
WL = Workload("s", T=2048, d=512, h=1024, E=4, k=2)


@pytest.fixture(scope="module")
def made():
    inp = {n: (v.cuda() if isinstance(v, torch.Tensor) else v) for n, v in I.layer_inputs(WL).items()}
    cfg = M.config_of(WL, train=True)
    W = M.pack_weights(cfg, inp["w1"], inp["w3"], inp["w2"])
    Wb = M.pack_weights_backward(cfg, inp["w1"], inp["w3"], inp["w2"])
    G = torch.randn((WL.T, WL.d), generator=torch.Generator(device="cuda").manual_seed(3),
                    device="cuda").bfloat16()
    torch.cuda.synchronize()
    return cfg, inp, W, Wb, G


def calls(made):
    """{name: call(stream) -> the tensors that it allocated and has to fill}"""
    cfg, g, W, Wb, G = made
    bufs = M.forward(cfg, g["x"], g["Wr"], g["bias"], *W)
    torch.cuda.synchronize()

    def backward(stream):
        r = M.backward(cfg, G, 0.1, g["x"], g["Wr"], g["bias"], *Wb, None, None, bufs, stream=stream)
        return [r[n] for n in ("dW13", "dW2p", "dx", "dWr")]

    def forward(stream):
        r = M.forward(cfg, g["x"], g["Wr"], g["bias"], *W, stream=stream)
        return [r[n] for n in ("out", "topk_idx", "topk_gate", "routed", "kept", "stats")]

    return {"pack": lambda s: list(M.pack_weights(cfg, g["w1"], g["w3"], g["w2"], stream=s)),
            "pack_backward": lambda s: list(M.pack_weights_backward(cfg, g["w1"], g["w3"], g["w2"],
                                                                    stream=s)),
            "forward": forward, "backward": backward}


@pytest.mark.parametrize("kind", ["stream", "address"])
@pytest.mark.parametrize("name", ["pack", "pack_backward", "forward", "backward"])
def test_results_on_a_given_stream(made, name, kind):
    call = calls(made)[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    arg = s if kind == "stream" else s.cuda_stream
    nbytes = [t.numel() * t.element_size() for t in want]
    # blocks of the results' sizes that the current stream still reads when they are freed
    torch.cuda.empty_cache()
    victims = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in nbytes]
    copies = [torch.zeros_like(v) for v in victims]
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    for c, v in zip(copies, victims):
        c.copy_(v)
    del victims, v
    got = call(arg)
    torch.cuda.synchronize()
    for c in copies:
        assert bool((c == 7).all())
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # results freed before the call has run: what is made of their blocks stays, and while
    # the stream is busy nothing is made of them
    del got, a, copies, c
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(CYCLES)
    got = call(arg)
    ptrs = {t.data_ptr() for t in got}
    del got
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in nbytes]
    taken = ptrs & {t.data_ptr() for t in junk}
    assert s.query() or not taken
    torch.cuda.synchronize()
    assert all(bool((t == 255).all()) for t in junk)
