"""The operators of a decode step, in their plain form and through the framework.

Four operators of the mixture-of-experts layer, told apart by a case's "op":

  few        the whole layer for 1 to 16 tokens, bf16 expert weights
  few_q4     the same with expert weights of 4 bits and one scale per group of
             32, 64 or 128 weights along the reduction
  quantize   packed bf16 expert weights to 4 bits; what comes back is the
             values that the 4 bits stand for
  dequantize 4-bit expert weights back to the packed bf16 layout

Weights are in the framework's packed layout: W13 [E][2h][d] holds, for each
block b of 128 hidden units, their gate rows at 256b .. 256b + 127 and their up
rows at 256b + 128 .. 256b + 255; W2p [E][d][h].  The shared experts are one
expert of width n_shared * h_shared in the same layout.
"""

import math

import torch

own = False


# ---------------------------------------------------------------- cases

def _layer(name, op, T, d, h, E, k, n_shared=0, h_shared=0, cf_num=0, cf_den=0, zipf=0.0,
           group=0):
    return {"name": name, "op": op, "T": T, "d": d, "h": h, "E": E, "k": k,
            "n_shared": n_shared, "h_shared": h_shared, "cf_num": cf_num, "cf_den": cf_den,
            "zipf": zipf, "group": group}


def _weights(name, op, d, h, E, group):
    return {"name": name, "op": op, "d": d, "h": h, "E": E, "group": group}


def listed():
    return [
        # one token through a tiny layer: launch and synchronisation latency alone
        _layer("few one token tiny", "few", 1, 128, 256, 8, 2),
        # one sequence decoding on the Mixtral-shaped layer of the decode workload
        _layer("few one token wide", "few", 1, 4096, 14336, 8, 2),
        # eight sequences on the layer with many small routed and two shared experts
        _layer("few eight many experts", "few", 8, 5120, 1536, 160, 6, 2, 1536),
        # an odd batch under a capacity limit and a skewed router: assignments drop,
        # popular experts see many tokens
        _layer("few thirteen capped", "few", 13, 1152, 2688, 12, 3, 0, 0, 5, 4, 1.0),
        # one sequence, 4-bit weights, the usual group of 128
        _layer("q4 one token wide", "few_q4", 1, 4096, 14336, 8, 2, group=128),
        # eight sequences, many experts, shared experts in 4 bits too
        _layer("q4 eight many experts", "few_q4", 8, 5120, 1536, 160, 6, 2, 1536, group=64),
        # the largest batch of the operator: every expert is hit, several tokens each
        _layer("q4 sixteen wide", "few_q4", 16, 4096, 14336, 8, 2, group=128),
        # odd sizes, the smallest group, capacity and a skewed router
        _layer("q4 three odd capped", "few_q4", 3, 640, 896, 5, 3, 1, 384, 3, 2, 0.5, group=32),
        # a small layer's weights, as a test or a draft model quantises them
        _weights("quantize small", "quantize", 640, 896, 5, 32),
        # the Mixtral-shaped layer's expert weights when a checkpoint is loaded
        _weights("quantize wide", "quantize", 4096, 14336, 8, 128),
        # a small layer brought back for a prefill
        _weights("dequantize small", "dequantize", 1152, 2688, 3, 64),
        # the Mixtral-shaped layer brought back for a prefill through the bf16 layer
        _weights("dequantize wide", "dequantize", 4096, 14336, 8, 128),
    ]


def _spread(rng, lo, hi, step=128):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["few", "few", "few_q4", "few_q4", "quantize", "dequantize"])
    E = int(round(math.exp(rng.uniform(math.log(2), math.log(160)))))
    d = _spread(rng, 128, 5120)
    # the whole expert set stays within that of the largest listed layers
    hmax = min(14336, int(3 * 10 ** 9 / (3 * d * E)) // 128 * 128)
    h = _spread(rng, 128, max(128, hmax))
    group = rng.choice([32, 64, 128])
    if op in ("quantize", "dequantize"):
        hmax = min(14336, int(1.4 * 10 ** 9 / (3 * d * E)) // 128 * 128)
        return {"op": op, "d": d, "h": min(h, max(128, hmax)), "E": E, "group": group}
    T = int(round(math.exp(rng.uniform(0.0, math.log(16)))))
    k = rng.randint(1, min(E, 8))
    n_shared = rng.choice([0, 0, 1, 2])
    h_shared = _spread(rng, 128, 2048) if n_shared else 0
    capped = rng.random() < 0.3
    c = _layer("", op, T, d, h, E, k, n_shared, h_shared, rng.choice([5, 6]) if capped else 0,
               4 if capped else 0, rng.choice([0.0, 0.0, 0.5, 1.2]),
               group if op == "few_q4" else 0)
    del c["name"]
    return c


def _hits(c):
    """Expected number of distinct experts that T tokens of k choices hit."""
    return c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])


def work(case):
    d, h, E = case["d"], case["h"], case["E"]
    if case["op"] in ("quantize", "dequantize"):
        n = 3.0 * d * h * E
        packed = n * (0.5 + 2.0 / case["group"])
        # quantize gives the values back as bf16, which reads the 4 bits again
        passes = 2 if case["op"] == "quantize" else 1
        return {"bytes": passes * (2.0 * n + packed), "flops": passes * n}
    T, k = case["T"], case["k"]
    hs = case["n_shared"] * case["h_shared"]
    per = 2.0 if case["op"] == "few" else 0.5 + 2.0 / case["group"]
    weights = 3.0 * d * (_hits(case) * h + hs)
    return {"bytes": weights * per + 4.0 * d * E + 4.0 * T * d,
            "flops": 6.0 * T * d * (k * h + hs) + 2.0 * T * d * E}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(gen, shape, std):
    """N(0, std^2) rounded to bf16, one expert at a time (the fp32 draw of a
    whole wide layer would not fit three times)."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for part in out:
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * std)
    return out


def _expert_weights(gen, n, d, h):
    """Packed W13 [n][2h][d] ~ N(0, 1/d) and W2p [n][d][h] ~ N(0, 1/h)."""
    return (_normal(gen, (n, 2 * h, d), 1.0 / math.sqrt(d)),
            _normal(gen, (n, d, h), 1.0 / math.sqrt(h)))


def _tokens(gen, c, Wr, bias):
    """x ~ N(0, 1) in bf16; tokens whose k + 1 best logits hold two within 1e-4
    of each other are drawn again, so that the choice of experts is one of the
    inputs' and not of a rounding."""
    x = torch.randn((c["T"], c["d"]), generator=gen, device="cuda").bfloat16()
    if c["E"] == 1:
        return x
    for _ in range(100):
        z = x.double() @ Wr.double() + bias.double()
        top = torch.sort(z, dim=1, descending=True).values[:, :min(c["k"] + 1, c["E"])]
        near = (top[:, :-1] - top[:, 1:]).amin(dim=1) < 1e-4
        if not bool(near.any()):
            break
        again = torch.randn(x.shape, generator=gen, device="cuda").bfloat16()
        x = torch.where(near[:, None], again, x)
    return x


def _codes(W, group):
    """4-bit codes (int8 in [-7, 7]) and scales (bf16) of rows along the last dim."""
    q = torch.empty(W.shape, dtype=torch.int8, device=W.device)
    s = torch.empty(W.shape[:-1] + (W.shape[-1] // group,), dtype=torch.bfloat16, device=W.device)
    for e in range(W.shape[0]):
        g = W[e].float().unflatten(-1, (-1, group))
        scale = (g.abs().amax(dim=-1) / 7.0).bfloat16()
        step = scale.float().unsqueeze(-1)
        code = torch.where(step > 0, torch.round(g / step), torch.zeros_like(g))
        q[e] = code.clamp(-7, 7).to(torch.int8).flatten(-2)
        s[e] = scale
    return q, s


def _config(c):
    import sparse_mixture_experts_22_b200 as M
    cf = (c["cf_num"], c["cf_den"]) if c.get("cf_den") else None
    return M.make_config(c.get("T", 1), c["d"], c["h"], c["E"], c.get("k", 1),
                         n_shared=c.get("n_shared", 0), h_shared=c.get("h_shared", 0), cf=cf,
                         has_bias=True)


def prepare(case, seed):
    c = dict(case)
    gen = _generator(seed)
    d, h, E, op = c["d"], c["h"], c["E"], c["op"]
    st = {"case": c}
    if op == "quantize":
        st["W13"], st["W2p"] = _expert_weights(gen, E, d, h)
        if own:
            st["cfg"] = _config(c)
        return st
    if op == "dequantize":
        W13, W2p = _expert_weights(gen, E, d, h)
        return _quantized(st, c, W13, W2p)
    st["Wr"] = torch.randn((d, E), generator=gen, device="cuda") / math.sqrt(d)
    # Zipf(s) popularity as the router's bias (zero without a skew)
    st["bias"] = -c["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda").float())
    st["x"] = _tokens(gen, c, st["Wr"], st["bias"])
    W13, W2p = _expert_weights(gen, E, d, h)
    shared = (_expert_weights(gen, 1, d, c["n_shared"] * c["h_shared"]) if c["n_shared"]
              else (None, None))
    if op == "few":
        st["W13"], st["W2p"], (st["W13s"], st["W2s"]) = W13, W2p, shared
        if own:
            import sparse_mixture_experts_22_b200 as M
            st["layer"] = M.FewLayer(_config(c), st["Wr"], st["bias"], W13, W2p, *shared)
        return st
    st = _quantized(st, c, W13, W2p, *shared)
    if own:
        import sparse_mixture_experts_22_b200 as M
        st["layer"] = M.FewLayer(_config(c), st["Wr"], st["bias"], *st["Q"], *st["Qs"],
                                 group=c["group"])
    return st


def _quantized(st, c, W13, W2p, W13s=None, W2s=None):
    """The 4-bit weights a program keeps: codes and scales here, the framework's
    packed form of the same ones there."""
    if own:
        import sparse_mixture_experts_22_b200 as M
        st["cfg"] = _config(c)
        st["Q"] = M.quantize_weights(st["cfg"], W13, W2p, c["group"])
        st["Qs"] = (M.quantize_weights(st["cfg"], W13s, W2s, c["group"], shared=True)
                    if W13s is not None else (None, None))
        return st
    st["c13"], st["c2"] = _codes(W13, c["group"]), _codes(W2p, c["group"])
    if W13s is not None:
        st["c13s"], st["c2s"] = _codes(W13s, c["group"]), _codes(W2s, c["group"])
    return st


# ---------------------------------------------------------------- plain forms

def _values(codes, group):
    """fp32 values of codes and scales (exact: 4 bits times 8)."""
    q, s = codes
    return (q.float().unflatten(-1, (-1, group)) * s.float().unsqueeze(-1)).flatten(-2)


def _gate_up(a):
    """[.., 2h] pre-activations in the packed interleave -> silu(gate) * up [.., h]."""
    b = a.unflatten(-1, (-1, 2, 128))
    gate, up = b[..., 0, :], b[..., 1, :]
    return (gate / (1.0 + torch.exp(-gate)) * up).flatten(-2)


def _plain_layer(st):
    c = st["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["group"]
    q4 = c["op"] == "few_q4"
    x = st["x"].float()
    z = x @ st["Wr"] + st["bias"]
    top, idx = torch.sort(z, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    gate = torch.exp(top - top[:, :1])
    gate = gate / gate.sum(dim=1, keepdim=True)
    chosen = torch.zeros((T, E), device="cuda").scatter_(1, idx, 1.0)
    routed = chosen.sum(dim=0)
    C = -(-T * k * c["cf_num"] // (E * c["cf_den"])) if c["cf_den"] else T
    rank = chosen.cumsum(dim=0) - chosen                   # earlier tokens of the expert
    kept = torch.clamp(routed, max=float(C))
    g = torch.zeros((T, E), device="cuda").scatter_(1, idx, gate) * (rank < C)

    def pick(name, codes, e):
        if not q4:
            return st[name][e].float()
        return _values((st[codes][0][e], st[codes][1][e]), G)

    if E <= T * k:      # every expert is read: all of them on all tokens, masked by the gate
        hid = _gate_up(torch.matmul(pick("W13", "c13", slice(None)), x.t()).transpose(1, 2))
        hid = hid * g.t().unsqueeze(-1)                    # [E][T][h]
        out = torch.matmul(hid, pick("W2p", "c2", slice(None)).transpose(1, 2)).sum(dim=0)
    else:               # the chosen experts' matrices, one copy per assignment
        e = idx.reshape(-1)
        xa = x.repeat_interleave(k, dim=0).unsqueeze(-1)
        hid = _gate_up(torch.matmul(pick("W13", "c13", e), xa).squeeze(-1))
        hid = (hid * g.gather(1, idx).reshape(-1, 1)).unsqueeze(-1)
        y = torch.matmul(pick("W2p", "c2", e), hid).squeeze(-1)
        out = y.unflatten(0, (T, k)).sum(dim=1)
    if c["n_shared"]:
        zero = torch.zeros(1, dtype=torch.long, device="cuda")
        hid = _gate_up(x @ pick("W13s", "c13s", zero)[0].t())
        out = out + hid @ pick("W2s", "c2s", zero)[0].t()
    return {"out": out.bfloat16(), "topk_idx": idx.int(), "topk_gate": gate,
            "routed": routed.int(), "kept": kept.int()}


def run(st):
    c = st["case"]
    op = c["op"]
    if own:
        import sparse_mixture_experts_22_b200 as M
        if op in ("few", "few_q4"):
            return st["layer"](st["x"])
        if op == "quantize":
            st["Q"] = M.quantize_weights(st["cfg"], st["W13"], st["W2p"], c["group"],
                                         out=st.get("Q"))
        st["back"] = M.dequantize_weights(st["cfg"], *st["Q"], c["group"], out=st.get("back"))
        return {"W13": st["back"][0], "W2p": st["back"][1]}
    if op in ("few", "few_q4"):
        return _plain_layer(st)
    if op == "quantize":
        return {"W13": torch.stack([_back(W, c["group"]) for W in st["W13"]]),
                "W2p": torch.stack([_back(W, c["group"]) for W in st["W2p"]])}
    return {"W13": _values(st["c13"], c["group"]).bfloat16(),
            "W2p": _values(st["c2"], c["group"]).bfloat16()}


def _back(W, group):
    """Rows of one expert quantised to 4 bits and back, rounded to bf16."""
    g = W.float().unflatten(-1, (-1, group))
    scale = (g.abs().amax(dim=-1, keepdim=True) / 7.0).bfloat16().float()
    code = torch.where(scale > 0, torch.round(g / scale).clamp(-7, 7), torch.zeros_like(g))
    return (code * scale).flatten(-2).bfloat16()


# ---------------------------------------------------------------- 64 bits

def _exact_quantized(W, group):
    """[rows][n] weights -> the 64-bit values their 4-bit codes stand for; the
    scale is part of the format and held in bf16."""
    rows, n = W.shape
    w = W.double().reshape(rows, n // group, group)
    amax = torch.maximum(w.max(dim=2).values, -w.min(dim=2).values)
    s = (amax / 7).to(torch.bfloat16).double()[:, :, None]
    ratio = w / torch.where(s == 0, torch.ones_like(s), s)
    q = torch.clamp(torch.round(ratio), min=-7, max=7)
    return torch.where(s == 0, torch.zeros_like(q), q * s).reshape(rows, n)


def _exact_ffn(v, W13, W2):
    """One expert, one token, in 64 bits."""
    a = (W13 @ v).reshape(-1, 256)
    gate, up = a[:, :128].reshape(-1), a[:, 128:].reshape(-1)
    return W2 @ (gate * torch.sigmoid(gate) * up)


def exact(case, seed):
    c, d, h, E, op = case, case["d"], case["h"], case["E"], case["op"]
    gen = _generator(seed)
    if op in ("quantize", "dequantize"):
        W13, W2p = _expert_weights(gen, E, d, h)
        return {"W13": torch.stack([_exact_quantized(W, c["group"]) for W in W13]),
                "W2p": torch.stack([_exact_quantized(W, c["group"]) for W in W2p])}
    T, k = c["T"], c["k"]
    Wr = torch.randn((d, E), generator=gen, device="cuda") / math.sqrt(d)
    bias = -c["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda").float())
    x = _tokens(gen, c, Wr, bias).double()
    W13, W2p = _expert_weights(gen, E, d, h)
    hs = c["n_shared"] * c["h_shared"]
    W13s, W2s = _expert_weights(gen, 1, d, hs) if hs else (None, None)
    w64 = (lambda W: _exact_quantized(W, c["group"])) if op == "few_q4" else (lambda W: W.double())
    z = (x @ Wr.double() + bias.double()).cpu()
    C = math.ceil(T * k * c["cf_num"] / (E * c["cf_den"])) if c["cf_den"] else T
    taken = [0] * E
    uses = {}
    idx, gates = torch.zeros((T, k), dtype=torch.int32), torch.zeros((T, k), dtype=torch.float64)
    for t in range(T):
        order = sorted(range(E), key=lambda e: (-float(z[t, e]), e))[:k]
        p = torch.softmax(z[t, order], dim=0)
        for j, e in enumerate(order):
            idx[t, j], gates[t, j] = e, p[j]
            if taken[e] < C:
                uses.setdefault(e, []).append((t, float(p[j])))
            taken[e] += 1
    out = torch.zeros((T, d), dtype=torch.float64, device="cuda")
    for e, tokens in uses.items():
        A, B = w64(W13[e]), w64(W2p[e])
        for t, p in tokens:
            out[t] += p * _exact_ffn(x[t], A, B)
    if hs:
        A, B = w64(W13s[0]), w64(W2s[0])
        for t in range(T):
            out[t] += _exact_ffn(x[t], A, B)
    routed = torch.tensor(taken, dtype=torch.int32)
    return {"out": out, "topk_idx": idx, "topk_gate": gates, "routed": routed,
            "kept": routed.clamp(max=C)}
