"""The few-token layer and 4-bit expert weights on the GPU, against the plain
64-bit form of few_check (which says what the tolerances are made of)."""

import math

import pytest
import torch

import few_check as F
import sparse_mixture_experts_22_b200 as M
from sparse_mixture_experts_22_b200 import inputs as I
from sparse_mixture_experts_22_b200.workloads import Workload

pytestmark = pytest.mark.gpu

CASES = {
    # one of everything
    "one": Workload("f_one", T=1, d=128, h=128, E=1, k=1),
    "tiny": Workload("f_tiny", T=1, d=128, h=256, E=8, k=2),
    # two parts of a token tile, model width in blocks of 128 that are no multiple of 256
    "full": Workload("f_full", T=16, d=384, h=384, E=6, k=3),
    # every token to the same experts
    "collapsed": Workload("f_coll", T=16, d=256, h=256, E=8, k=2, zipf_s=40.0),
    "eight_same": Workload("f_eight", T=8, d=640, h=256, E=3, k=3),
    # assignments drop; in the second almost all of them, leaving tokens without an expert
    "capped": Workload("f_cap", T=13, d=256, h=384, E=4, k=2, cf=(5, 4), zipf_s=1.0),
    "starved": Workload("f_starved", T=12, d=128, h=128, E=4, k=1, cf=(1, 12), zipf_s=3.0),
    "shared": Workload("f_shared", T=9, d=512, h=256, E=5, k=2, n_shared=2, h_shared=128),
    "many": Workload("f_many", T=7, d=640, h=128, E=160, k=6, n_shared=1, h_shared=384),
    # as many experts as a batch can hit
    "widest": Workload("f_widest", T=16, d=128, h=128, E=1024, k=8),
    # more hidden units than the parts hold at once
    "long_h": Workload("f_long_h", T=11, d=128, h=10240, E=8, k=8),
    "long_d": Workload("f_long_d", T=2, d=8192, h=128, E=2, k=1),
    # many stages a granule and several granules a part, experts of very different loads
    "uneven": Workload("f_uneven", T=16, d=2048, h=1024, E=7, k=3, n_shared=1, h_shared=512,
                       zipf_s=1.5),
    "deep": Workload("f_deep", T=6, d=4096, h=1408, E=4, k=4),
}

_made = {}


def made(name, group=0):
    """(workload, host inputs, 64-bit reference) of a case, group 0 for bf16."""
    if (name, group) not in _made:
        wl = CASES[name]
        inp = I.layer_inputs(wl)
        w = {n: inp[n] for n in ("w1", "w3", "w2", "w1s", "w3s", "w2s") if n in inp}
        if group:
            # groups run along the reduction: d for w1 and w3, the hidden width for w2
            # (the shared experts' hidden units laid end to end: multiples of 128 each)
            w = {n: F.quantize(v.transpose(1, 2), group)[2].transpose(1, 2) for n, v in w.items()}
        shared = (w["w1s"], w["w3s"], w["w2s"]) if wl.n_shared else None
        ref = F.layer(inp["x"], inp["Wr"], inp["bias"], wl.k, w["w1"], w["w3"], w["w2"], shared,
                      wl.cf, group > 0)
        _made[name, group] = (wl, inp, ref)
    return _made[name, group]


def device_weights(wl, inp, dev="cuda"):
    cfg = M.config_of(wl)
    g = {n: (v.to(dev) if isinstance(v, torch.Tensor) else v) for n, v in inp.items()}
    W = list(M.pack_weights(cfg, g["w1"], g["w3"], g["w2"]))
    W += list(M.pack_weights(cfg, g["w1s"], g["w3s"], g["w2s"], shared=True)) if wl.n_shared else []
    return cfg, g, W


def make_layer(wl, inp, group=0, **kw):
    cfg, g, W = device_weights(wl, inp)
    if group:
        W = [*M.quantize_weights(cfg, *W[:2], group),
             *(M.quantize_weights(cfg, *W[2:], group, shared=True) if W[2:] else ())]
    W += [None] * (4 - len(W))
    return M.FewLayer(cfg, g["Wr"], g["bias"], *W, group=group or None, **kw), g


def run(layer, x):
    got = layer(x)
    torch.cuda.synchronize()
    assert M.moe_read_device_status(layer.ws) == 0
    return got


# ---------------------------------------------------------------- 4-bit weights

@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 128, 128), (3, 384, 640), (2, 256, 1152)])
def test_quantized_values(shape, group):
    """Codes and scales are the formula's, bit for bit: the values read back are
    q s rounded once to bf16."""
    E, d, h = shape
    cfg = M.make_config(1, d, h, E, 1)
    gen = torch.Generator().manual_seed(E + group)
    W13 = (torch.randn((E, 2 * h, d), generator=gen) / math.sqrt(d)).bfloat16()
    W2p = (torch.randn((E, d, h), generator=gen) / math.sqrt(h)).bfloat16()
    W13[0, 3] = 0                       # groups without a scale
    W2p[0, 1, :group] = 0
    W13[0, 5, :group] *= 1e-3           # a group of another magnitude
    W2p[-1, -1, -1] = 8.0               # an outlier: the rest of its group rounds to 0
    W13[0, 7, 0] = 1e-38                # a scale near the end of the range
    W13[0, 7, 1:group] = 0
    Q = M.quantize_weights(cfg, W13.cuda(), W2p.cuda(), group)
    back = M.dequantize_weights(cfg, *Q, group)
    torch.cuda.synchronize()
    for got, W in zip(back, (W13, W2p)):
        q, s, v = F.quantize(W, group)
        assert torch.equal(got.cpu(), v.float().bfloat16())


def test_quantized_shared_set_and_reuse():
    wl = CASES["shared"]
    cfg, g, W = device_weights(wl, I.layer_inputs(wl))
    out = M.quantize_weights(cfg, *W[2:], 64, shared=True)
    again = tuple(torch.full_like(q, 255) for q in out)
    assert M.quantize_weights(cfg, *W[2:], 64, shared=True, out=again) is again
    back = M.dequantize_weights(cfg, *again, 64, shared=True)
    torch.cuda.synchronize()
    for a, b in zip(out, again):
        assert torch.equal(a, b)
    for got, w in zip(back, W[2:]):
        assert torch.equal(got.cpu(), F.quantize(w.cpu(), 64)[2].float().bfloat16())


def test_quantize_writes_its_buffers_only():
    cfg = M.make_config(1, 256, 384, 3, 1)
    W13 = torch.randn((3, 768, 256), device="cuda").bfloat16()
    W2p = torch.randn((3, 256, 384), device="cuda").bfloat16()
    n13, n2 = M.moe_q4_size(cfg, 0, 32)
    guard = [torch.full((n + 512,), 170, dtype=torch.uint8, device="cuda") for n in (n13, n2)]
    q = (guard[0][256:256 + n13], guard[1][256:256 + n2])
    M.quantize_weights(cfg, W13, W2p, 32, out=q)
    flat = [torch.full((W.numel() + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
            for W in (W13, W2p)]
    back = tuple(f[128:-128].view(W.shape) for f, W in zip(flat, (W13, W2p)))
    M.dequantize_weights(cfg, *q, 32, out=back)
    torch.cuda.synchronize()
    for b in guard:
        assert bool((b[:256] == 170).all()) and bool((b[-256:] == 170).all())
    for f in flat:
        assert bool((f[:128] == 7).all()) and bool((f[-128:] == 7).all())
    for b, W in zip(back, (W13, W2p)):
        assert torch.equal(b.cpu(), F.quantize(W.cpu(), 32)[2].float().bfloat16())


# ---------------------------------------------------------------- the layer

@pytest.mark.parametrize("name", list(CASES))
def test_few_layer(name):
    wl, inp, ref = made(name)
    layer, g = make_layer(wl, inp)
    layer.ws.fill_(0xFF)                 # nothing of the workspace is taken as it was found
    got = run(layer, g["x"])
    F.check(got, ref)
    first = {n: v.clone() for n, v in got.items()}
    for _ in range(2):                   # the same bits again
        for n, v in run(layer, g["x"]).items():
            assert torch.equal(v, first[n]), n


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("name", list(CASES))
def test_few_layer_q4(name, group):
    wl, inp, ref = made(name, group)
    layer, g = make_layer(wl, inp, group)
    layer.ws.fill_(0xFF)
    got = run(layer, g["x"])
    F.check(got, ref)
    first = {n: v.clone() for n, v in got.items()}
    for n, v in run(layer, g["x"]).items():
        assert torch.equal(v, first[n]), n


def test_starved_tokens_get_zero():
    wl, inp, ref = made("starved")
    layer, g = make_layer(wl, inp)
    got = run(layer, g["x"])
    empty = ref["out"].abs().amax(1) == 0
    assert int(empty.sum()) >= 6
    assert bool((got["out"].cpu()[empty] == 0).all())


@pytest.mark.parametrize("group", [0, 128])
def test_every_batch_size_of_one_layer(group):
    """One FewLayer serves every batch up to its size; a batch's rows behind the
    last token stay as they were."""
    wl, inp, _ = made("full", group)
    layer, g = make_layer(wl, inp, group)
    whole = run(layer, g["x"])["out"].clone()
    for t in (0, 1, 2, 7, 8, 9, 15, 16):
        layer.bufs["out"].fill_(5.0)
        got = run(layer, g["x"][:t].contiguous())
        assert got["out"].shape == (t, wl.d) and got["topk_idx"].shape == (t, wl.k)
        assert int(got["routed"].sum()) == t * wl.k
        # without a capacity limit a token's output does not depend on the others
        # but for the order of its partial sums
        diff = (got["out"].float() - whole[:t].float()).abs()
        assert bool((diff <= 2.0 ** -7 * whole[:t].float().abs() + 1e-5).all())
        assert bool((layer.bufs["out"][t:] == 5.0).all())


@pytest.mark.parametrize("name", ["shared", "capped"])
def test_routing_and_output_beside_the_whole_layer(name):
    """The same routing as moe_forward, and the same output to a bf16 rounding."""
    wl, inp, _ = made(name)
    cfg, g, W = device_weights(wl, inp)
    W += [None] * (4 - len(W))
    cfg_s = M.config_of(wl, hidden="split")
    full = M.forward(cfg_s, g["x"], g["Wr"], g["bias"], *W)
    layer = M.FewLayer(cfg, g["Wr"], g["bias"], *W, with_stats=True)
    got = run(layer, g["x"])
    for n in ("topk_idx", "routed", "kept"):
        assert torch.equal(got[n], full[n]), n
    a, b = got["out"].float(), full["out"].float()
    # two roundings to bf16 of values that differ by fp32 sums only
    assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-4).all())
    s, f = M.stats_dict(got["stats"]), M.stats_dict(full["stats"])
    assert s["tokens"] == f["tokens"] and s["dropped"] == f["dropped"]
    for n in ("aux_loss", "overflow_rate", "mean_entropy"):
        assert abs(s[n] - f[n]) <= 1e-5 * abs(f[n]), n


@pytest.mark.parametrize("group", [0, 64])
def test_a_token_of_nan_stays_alone(group):
    wl, inp, ref = made("shared", group)
    layer, g = make_layer(wl, inp, group)
    clean = run(layer, g["x"])["out"].clone()
    x = g["x"].clone()
    x[4] = float("nan")
    got = run(layer, x)
    assert bool(got["out"][4].isnan().all())
    # NaN logits count as -inf: the lowest experts, whatever the others chose
    assert got["topk_idx"][4].cpu().tolist() == list(range(wl.k))
    others = [t for t in range(wl.T) if t != 4]
    diff = (got["out"][others].float() - clean[others].float()).abs()
    assert bool((diff <= 2.0 ** -7 * clean[others].float().abs() + 1e-5).all())


@pytest.mark.parametrize("group", [0, 32])
def test_tokens_of_very_different_size(group):
    """Each row is scaled by itself: neither the largest nor the smallest token moves
    the others out of their bounds."""
    wl = Workload("f_scale", T=4, d=256, h=128, E=2, k=2)
    inp = I.layer_inputs(wl)
    inp["x"] = (inp["x"].double() * torch.tensor([[2.0 ** -60], [2.0 ** -20], [2.0 ** 20],
                                                  [2.0 ** 50]])).to(torch.bfloat16)
    w = {n: F.quantize(inp[n].transpose(1, 2), group)[2].transpose(1, 2) if group else inp[n]
         for n in ("w1", "w3", "w2")}
    ref = F.layer(inp["x"], inp["Wr"], None, wl.k, w["w1"], w["w3"], w["w2"], None, None, group > 0)
    layer, g = make_layer(wl, inp, group)
    F.check(run(layer, g["x"]), ref)


def test_stats_of_an_empty_batch():
    wl, inp, _ = made("full")
    layer, g = make_layer(wl, inp, with_stats=True)
    run(layer, g["x"])
    got = run(layer, g["x"][:0])
    cfg, _, W = device_weights(wl, inp)
    cfg = M.config_of(wl, T=0)
    want = M.forward(cfg, g["x"][:0], g["Wr"], g["bias"], *W)
    torch.cuda.synchronize()
    assert torch.equal(got["stats"], want["stats"])
    assert int(got["routed"].abs().sum()) == 0 and int(got["kept"].abs().sum()) == 0


def test_experts_masked_by_their_bias():
    """-inf and the type's lowest value in the bias keep experts from being chosen."""
    wl, inp, _ = made("capped")
    inp = dict(inp)
    for low in (float("-inf"), torch.finfo(torch.float32).min):
        inp["bias"] = torch.tensor([low, 0.0, low, 0.1])
        layer, g = make_layer(wl, inp)
        got = run(layer, g["x"])
        ref = F.layer(inp["x"], inp["Wr"], inp["bias"], wl.k, inp["w1"], inp["w3"], inp["w2"],
                      None, wl.cf)
        F.check(got, ref)
        assert got["routed"].cpu().tolist() == [0, wl.T, 0, wl.T]


@pytest.mark.parametrize("group", [0, 32])
def test_unread_experts_may_hold_nan(group):
    """Only the experts a batch hits are read."""
    wl, inp, ref = made("tiny", group)
    hit = set(ref["idx"].flatten().tolist())
    layer, g = make_layer(wl, inp, group)
    for e in range(wl.E):
        if e not in hit:
            for w in layer._held[2:4]:
                if group and w is layer._held[2]:
                    # blocks of codes and their scales: all bits set make the scales NaN
                    w.view(wl.E, -1)[e] = 255
                elif group:
                    # the codes of every expert come first, then the scales of every expert
                    codes = wl.E * (wl.d // 128) * (wl.h // 32) * 2048
                    w[codes:].view(wl.E, -1)[e] = 255
                else:
                    w[e] = float("nan")
    F.check(run(layer, g["x"]), ref)


@pytest.mark.parametrize("group", [0, 128])
def test_graph_replay_gives_the_eager_bits(group):
    wl, inp, ref = made("many", group)
    layer, g = make_layer(wl, inp, group, with_stats=True)
    eager = {n: v.clone() for n, v in run(layer, g["x"]).items()}
    other = torch.randn_like(g["x"].float()).bfloat16()
    x = other.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        layer(x)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            layer(x)
    torch.cuda.synchronize()
    x.copy_(g["x"])                      # a replay takes the inputs as they are then
    for _ in range(2):
        for v in layer.bufs.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, v in eager.items():
            assert torch.equal(layer.bufs[n], v), n
    del graph


@pytest.mark.parametrize("pdl", [True, False])
@pytest.mark.parametrize("group", [0, 32])
def test_steps_right_behind_what_they_read(group, pdl):
    """Weights, x and the workspace are written by the work just before a call, and a
    step's output is the next one's input: eager, and captured behind a copy and a
    join with another stream."""
    wl = Workload("f_chain", T=5, d=256, h=256, E=6, k=2, n_shared=1, h_shared=128)
    inp = I.layer_inputs(wl)
    cfg, g, W = device_weights(wl, inp)
    if group:
        sets = [M.quantize_weights(cfg, *W[:2], group),
                M.quantize_weights(cfg, *W[2:], group, shared=True)]
        W = [*sets[0], *sets[1]]
    layers = [M.FewLayer(cfg, g["Wr"], None, *[torch.zeros_like(w) for w in W], group=group or None)
              for _ in range(3)]
    x = torch.zeros_like(g["x"])

    def steps():
        x.copy_(g["x"])
        y = x
        for layer in layers:
            for own, w in zip(layer._held[2:], W):
                own.copy_(w)
            y = layer(y)["out"]
        return y

    def clear():
        x.zero_()
        for layer in layers:
            layer.bufs["out"].zero_()
            for own in layer._held[2:]:
                own.zero_()
            layer.ws.fill_(255)
        torch.cuda.synchronize()

    want = g["x"]
    for layer in layers:  # one at a time
        for own, w in zip(layer._held[2:], W):
            own.copy_(w)
        torch.cuda.synchronize()
        want = run(layer, want)["out"].clone()
    assert torch.isfinite(want.float()).all() and want.float().abs().max() > 0
    M.moe_set_pdl(pdl)
    try:
        for _ in range(3):
            clear()
            got = steps()
            torch.cuda.synchronize()
            assert torch.equal(got, want)
        s, side = torch.cuda.Stream(), torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            side.wait_stream(s)
            with torch.cuda.stream(side):
                for layer in layers:
                    layer.bufs["routed"].zero_()
            s.wait_stream(side)
            got = steps()
        for _ in range(3):
            clear()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want)
        del graph
    finally:
        M.moe_set_pdl(True)


def test_two_layers_on_two_streams():
    """Calls of layers with their own workspaces may overlap."""
    made_ = [(*made(n, q), q) for n, q in (("many", 0), ("full", 64))]
    layers = [make_layer(wl, inp, q) for wl, inp, _, q in made_]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(20):
        for (layer, g), s in zip(layers, streams):
            layer(g["x"], stream=s)
    torch.cuda.synchronize()
    for (layer, _), (_, _, ref, _) in zip(layers, made_):
        assert M.moe_read_device_status(layer.ws) == 0
        F.check(layer.bufs, ref)


def test_prefill_then_decode_from_the_same_4_bits():
    """Quantise once; a prefill of 40 tokens through the read-back weights and
    moe_forward, then decode steps of 3 tokens through the 4-bit layer."""
    G = 64
    wl = Workload("f_serve", T=43, d=384, h=256, E=6, k=2, n_shared=1, h_shared=256)
    inp = I.layer_inputs(wl)
    cfg, g, W = device_weights(wl.scaled(T=3), inp)
    Q = M.quantize_weights(cfg, *W[:2], G)
    Qs = M.quantize_weights(cfg, *W[2:], G, shared=True)
    back = [*M.dequantize_weights(cfg, *Q, G), *M.dequantize_weights(cfg, *Qs, G, shared=True)]
    names = ("w1", "w3", "w2", "w1s", "w3s", "w2s")
    w = {n: F.quantize(inp[n].transpose(1, 2), G)[2].transpose(1, 2) for n in names}
    pre = M.forward(M.config_of(wl, T=40, hidden="split"), g["x"][:40].contiguous(), g["Wr"], None,
                    *back)
    torch.cuda.synchronize()
    wb = {n: v.float().bfloat16() for n, v in w.items()}
    ref = F.layer(inp["x"][:40], inp["Wr"], None, wl.k, wb["w1"], wb["w3"], wb["w2"],
                  (wb["w1s"], wb["w3s"], wb["w2s"]))
    F.check(pre, ref)
    layer = M.FewLayer(cfg, g["Wr"], None, *Q, *Qs, group=G)
    for at in (40, 20, 0):
        x = inp["x"][at:at + 3]
        ref = F.layer(x, inp["Wr"], None, wl.k, w["w1"], w["w3"], w["w2"],
                      (w["w1s"], w["w3s"], w["w2s"]), None, True)
        F.check(run(layer, x.cuda()), ref)


@pytest.mark.parametrize("group", [0, 64])
def test_a_wait_that_runs_out_is_reported(group):
    """The test hook keeps block 0 from bringing anything in: its bounded waits
    run out, the status says so, and the next call is as before."""
    wl, inp, ref = made("full", group)
    layer, g = make_layer(wl, inp, group)
    want = run(layer, g["x"])["out"].clone()
    M.moe_set_wait_limit_ns(5_000_000)
    M.binding.moe_set_test_stall(True)
    try:
        layer(g["x"])
        status = M.moe_read_device_status(layer.ws)
    finally:
        M.binding.moe_set_test_stall(False)
        M.moe_set_wait_limit_ns(2_000_000_000)
    assert status == 7
    assert torch.equal(run(layer, g["x"])["out"], want)


def test_launch_count_of_a_decode_step():
    wl, inp, _ = made("shared")
    layer, g = make_layer(wl, inp)
    run(layer, g["x"])
    n = M.moe_launch_count()
    layer(g["x"])
    assert 1 <= M.moe_launch_count() - n <= 3
    torch.cuda.synchronize()
