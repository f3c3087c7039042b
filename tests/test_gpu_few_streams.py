"""4-bit conversions and the few-token layer on given streams: no call writes memory
that another stream still reads, and no memory is handed out again under a call.

A stream is held up by a kernel that only waits some 20 ms.  The caching allocator hands
a block freed on the current stream out again at once; one that another stream was
recorded on only after that stream is done."""

import pytest
import torch

import few_check as F
import sparse_mixture_experts_22_b200 as M
from test_gpu_few import device_weights, made, make_layer

pytestmark = pytest.mark.gpu

GROUP = 64
CYCLES = 40_000_000


@pytest.fixture
def packed():
    E, d, h = 3, 1024, 1024
    gen = torch.Generator(device="cuda").manual_seed(1)
    W13 = torch.randn((E, 2 * h, d), generator=gen, device="cuda").bfloat16()
    W2p = torch.randn((E, d, h), generator=gen, device="cuda").bfloat16()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    return M.make_config(1, d, h, E, 1), W13, W2p


def want(W):
    return F.quantize(W.cpu(), GROUP)[2].float().bfloat16()


def as_stream(kind):
    s = torch.cuda.Stream()
    return s, (s if kind == "stream" else s.cuda_stream)


def read_while_freed(size):
    """Frees blocks of `size` bytes of sevens that the current stream has yet to copy."""
    victims = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
    copies = [torch.zeros_like(v) for v in victims]
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    for c, v in zip(copies, victims):
        c.copy_(v)
    return copies


@pytest.mark.parametrize("kind", ["stream", "address"])
@pytest.mark.parametrize("op", ["quantize", "dequantize"])
def test_result_waits_for_its_memory(packed, op, kind):
    """The current stream still reads the block that the result is put in."""
    cfg, W13, W2p = packed
    s, arg = as_stream(kind)
    Q = M.quantize_weights(cfg, W13, W2p, GROUP)
    if op == "quantize":
        call, size = (lambda: M.quantize_weights(cfg, W13, W2p, GROUP, stream=arg)), Q[0].numel()
    else:
        call, size = (lambda: M.dequantize_weights(cfg, *Q, GROUP, stream=arg)), W13.numel() * 2
    copies = read_while_freed(size)
    got = call()
    torch.cuda.synchronize()
    assert all(bool((c == 7).all()) for c in copies)
    back = got if op == "dequantize" else M.dequantize_weights(cfg, *got, GROUP)
    for b, W in zip(back, (W13, W2p)):
        assert torch.equal(b.cpu(), want(W))


@pytest.mark.parametrize("kind", ["stream", "address"])
@pytest.mark.parametrize("op", ["quantize", "dequantize"])
def test_memory_is_kept_until_the_call_is_done(packed, op, kind):
    """Inputs and results freed while the given stream has yet to come to the call."""
    cfg, W13, W2p = packed
    s, arg = as_stream(kind)
    Q = M.quantize_weights(cfg, W13, W2p, GROUP)
    torch.cuda.synchronize()
    src = [t.clone() for t in ((W13, W2p) if op == "quantize" else Q)]
    ins = [(t.data_ptr(), t.numel() * t.element_size()) for t in src]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(CYCLES)
    fn = M.quantize_weights if op == "quantize" else M.dequantize_weights
    kept = fn(cfg, *src, GROUP, stream=arg)
    lost = fn(cfg, *src, GROUP, stream=arg)
    outs = [(t.data_ptr(), t.numel() * t.element_size()) for t in lost]
    del src, lost
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _, n in ins + outs]
    taken = {t.data_ptr() for t in junk} & {p for p, _ in ins + outs}
    assert s.query() or not taken
    torch.cuda.synchronize()
    assert all(bool((t == 255).all()) for t in junk)
    back = kept if op == "dequantize" else M.dequantize_weights(cfg, *kept, GROUP)
    for b, W in zip(back, (W13, W2p)):
        assert torch.equal(b.cpu(), want(W))


@pytest.mark.parametrize("group", [0, 64])
def test_layer_waits_for_its_memory(group):
    """The constructor's stream still reads the blocks that the layer's buffers are put
    in, and the first call comes on another stream."""
    wl, inp, ref = made("uneven", group)
    layer, g = make_layer(wl, inp, group)
    weights = layer._held
    need = layer.ws.numel()
    torch.cuda.synchronize()
    del layer
    torch.cuda.empty_cache()
    copies = read_while_freed(need)
    layer = M.FewLayer(M.config_of(wl), *weights, group=group or None)
    got = layer(g["x"], stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(bool((c == 7).all()) for c in copies)
    F.check(got, ref)


@pytest.mark.parametrize("kind", ["stream", "address"])
@pytest.mark.parametrize("group", [0, 64])
def test_layer_memory_is_kept_until_the_call_is_done(group, kind):
    """x, the layer and its weights freed while the given stream has yet to come to the
    call; what is made in the meantime keeps its values."""
    wl, inp, ref = made("uneven", group)
    s, arg = as_stream(kind)
    layer, g = make_layer(wl, inp, group)
    x = g["x"].clone()
    first = layer(g["x"], stream=arg)
    torch.cuda.synchronize()
    F.check(first, ref)
    first = {n: v.clone() for n, v in first.items()}
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(CYCLES)
    out = layer(x, stream=arg)["out"]
    with torch.cuda.stream(s):
        result = out.clone()
    blocks = [t for t in (*layer._held, layer.ws, x) if t is not None]
    sizes = [t.numel() * t.element_size() for t in blocks]
    ptrs = {t.data_ptr() for t in blocks}
    del blocks, layer, x, out, g
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
    taken = ptrs & {t.data_ptr() for t in junk}
    assert s.query() or not taken
    torch.cuda.synchronize()
    assert all(bool((t == 255).all()) for t in junk)
    assert torch.equal(result, first["out"])


@pytest.mark.parametrize("group", [0, 64])
def test_layer_made_inside_a_capture(group):
    """A layer may be made while its stream is being captured; the graph's pool holds
    its buffers."""
    wl, inp, ref = made("shared", group)
    cfg, g, W = device_weights(wl, inp)
    if group:
        W = [*M.quantize_weights(cfg, *W[:2], group), *M.quantize_weights(cfg, *W[2:], group, shared=True)]
    warm = M.FewLayer(cfg, g["Wr"], g["bias"], *W, group=group or None)
    warm(g["x"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer = M.FewLayer(cfg, g["Wr"], g["bias"], *W, group=group or None)
        got = layer(g["x"])
    graph.replay()
    torch.cuda.synchronize()
    F.check(got, ref)
    del graph
