"""A plain 64-bit form of the few-token layer and of 4-bit weights, with a bound
on what fp32 sums and the stated roundings may move each output.

bound[t][c] adds up, per element:
  2^-8 |out|                         the bf16 store (half of eps = 2^-7)
  GATE_ABS sum_j |y_j|               gates off by at most GATE_ABS (fp32 logits)
  sum |g w2| dH                      the hidden activations, where
      dH = 2^-17 |H|                 stored as two bf16 parts (2^-9 of 2^-8 of H)
         + 1.1 |up| da + |silu| du   |silu'| <= 1.1; 2^-20 |H| for silu's own fp32 steps
      da = n_d 2^-23 sum |x w1|      fp32 sums of d products in steps of 16, eight
                                     partial sums (n_d = d / 16 + 16; tensor-core
                                     adds truncate: one 2^-23 each), du alike
  n_h 2^-23 sum |g H w2|             the down sum, in steps of 16 with two parts
                                     each (n_h = 2 h / 16 + parts)

With 4-bit weights the products and the sums of a group are exact, and x and H are
integers times a power of two instead: of a row of x, the largest magnitude lies
in [2^21, 2^22) units, so that rounding moves an element by half a unit, 2^-22 of
the largest at most; of g H the same within an expert's share of a part.  So
      dx = 2^-22 max |x|,  da gains dx sum |w1|,  du likewise
      dH = 2^-22 max |H|             in place of 2^-17 |H|
(both bounds are kept, added up: the sums over groups are in fp32 as before).
"""

import torch

GATE_ABS = 2.5e-5


def quantize(w, group):
    """[..., n] weights -> (codes, bf16 scales, fp64 values)."""
    g = w.float().unflatten(-1, (-1, group))
    s = (g.abs().amax(-1, keepdim=True) / 7.0).to(torch.bfloat16)
    f = s.float()
    q = torch.where(f > 0, torch.round(g / torch.where(f > 0, f, torch.ones_like(f))),
                    torch.zeros_like(g)).clamp(-7, 7)
    return q.flatten(-2), s.squeeze(-1), (q.double() * s.double()).flatten(-2)


def _ffn(x, w1, w3, w2, g, q4):
    """One expert on one token: (g * ffn(x), its bound without the gate's error)."""
    d, h = w1.shape
    a, u = x @ w1, x @ w3
    dx = 2.0 ** -22 * x.abs().max() if q4 else 0.0
    da = (d / 16 + 16) * 2.0 ** -23 * (x.abs() @ w1.abs()) + dx * w1.abs().sum(0)
    du = (d / 16 + 16) * 2.0 ** -23 * (x.abs() @ w3.abs()) + dx * w3.abs().sum(0)
    s = a * torch.sigmoid(a)
    H = s * u
    stored = 2.0 ** -22 * H.abs().max() if q4 else 2.0 ** -17 * H.abs()
    dH = stored + 2.0 ** -20 * H.abs() + 1.1 * u.abs() * da + s.abs() * du
    y = H @ w2
    dy = dH @ w2.abs() + (2 * h / 16 + 300) * 2.0 ** -23 * (H.abs() @ w2.abs())
    return g * y, g * dy, y.abs()


def layer(x, Wr, bias, k, w1, w3, w2, shared=None, cf=None, q4=False):
    """x [T][d]; w1, w3 [E][d][h], w2 [E][h][d] (any float type); shared: (w1s,
    w3s, w2s) of [S] experts; q4: bounds of the 4-bit form.  Returns a dict with out, bound, idx, gate,
    routed, kept in fp64 / ints."""
    x, Wr = x.double(), Wr.double()
    T, E = x.shape[0], Wr.shape[1]
    z = x @ Wr + (bias.double() if bias is not None else 0.0)
    C = T if cf is None else -(-T * k * cf[0] // (E * cf[1]))
    routed = [0] * E
    idx = torch.zeros((T, k), dtype=torch.int64)
    gate = torch.zeros((T, k), dtype=torch.float64)
    out = torch.zeros_like(x)
    bound = torch.zeros_like(x)
    for t in range(T):
        order = sorted(range(E), key=lambda e: (-float(z[t, e]), e))[:k]
        p = torch.softmax(z[t, order], 0)
        for j, e in enumerate(order):
            idx[t, j], gate[t, j] = e, p[j]
            routed[e] += 1
            if routed[e] <= C:
                y, dy, ya = _ffn(x[t], w1[e].double(), w3[e].double(), w2[e].double(), p[j], q4)
                out[t] += y
                bound[t] += dy + GATE_ABS * ya
        for s in range(shared[0].shape[0] if shared else 0):
            y, dy, _ = _ffn(x[t], *(w[s].double() for w in shared), 1.0, q4)
            out[t] += y
            bound[t] += dy
    bound += 2.0 ** -8 * (out.abs() + bound)
    return {"out": out, "bound": bound, "idx": idx, "gate": gate, "routed": routed,
            "kept": [min(r, C) for r in routed]}


def check(got, ref):
    """Outputs of one call against layer()'s."""
    assert torch.equal(got["topk_idx"].cpu().long(), ref["idx"])
    assert (got["topk_gate"].cpu().double() - ref["gate"]).abs().max() <= GATE_ABS
    assert got["routed"].cpu().tolist() == ref["routed"]
    assert got["kept"].cpu().tolist() == ref["kept"]
    err = (got["out"].cpu().double() - ref["out"]).abs()
    worst = (err - ref["bound"]).max()
    assert bool((err <= ref["bound"]).all()), f"worst excess over the bound {float(worst)}"
