"""Plain 64-bit statements of the routing from given logits (k3moe_gate) and
of the dense product (k3moe_linear), and the error bounds that the kernels'
arithmetic has against them.  numpy / torch on whatever device the inputs are;
nothing here is shared with the library."""
from __future__ import annotations

import math

import numpy as np

NONE = -np.inf


def gate_ref(logits, k, score="softmax", bias=None, groups=1, kept=1, group_top=1, renorm=False, scale=1.0):
    """-> (idx int32 [T, k], weight float64 [T, k]) of fp64 logits [T, E]."""
    T, E = logits.shape
    size = E // groups
    idx = np.full((T, k), -1, dtype=np.int32)
    weight = np.zeros((T, k))
    for t in range(T):
        l = [float(v) for v in logits[t]]
        if score == "sigmoid":
            s = [1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 if v == v else math.nan for v in l]
        elif any(v != v or v == math.inf for v in l):
            s = [math.nan] * E
        else:
            m = max(l)
            e = [math.exp(v - m) if v > NONE else 0.0 for v in l]
            z = math.fsum(e)
            s = [v / z if z else 0.0 for v in e]
        c = [s[e] + float(bias[e]) if bias is not None else s[e] for e in range(E)]
        rank = c if bias is not None else l
        live = [e for e in range(E) if l[e] > NONE and rank[e] > NONE]  # NaN compares false
        if groups > 1 and kept < groups:
            # one value ranks by the logits where there is no bias, two are a sum of scores
            val = rank if group_top == 1 else c
            tot = []
            for g in range(groups):
                mine = sorted((val[e] if val[e] > NONE else NONE for e in live if e // size == g), reverse=True)
                mine = mine[:group_top]
                tot.append(sum(mine) if len(mine) == group_top and min(mine) > NONE else NONE)
            stay = set(sorted(range(groups), key=lambda g: (-tot[g], g))[:kept])
            live = [e for e in live if e // size in stay]
        pick = sorted(live, key=lambda e: (-rank[e], e))[:k]
        w = [s[e] for e in pick]
        z = sum(w)
        for j, e in enumerate(pick):
            idx[t, j] = e
            weight[t, j] = scale * ((w[j] / z if z != 0 else 0.0) if renorm else w[j])
    return idx, weight


# Weights against gate_ref: the score of a pick comes from an exponential (2
# units in the last place of fp32), its argument l - max rounded once (at most
# x e^-x <= 0.37 of a unit in the sum, none in a pick's own 64-bit score) and a
# sum of at most 32 + 5 additions, half a unit each; then at most four more
# roundings (score, sum of the picks, quotient, scale): 64 half units in all.
GATE_RTOL = 64 * 2.0 ** -24
GATE_ATOL = 2.0 ** -126  # below fp32's normal range


def act64(v, kind):
    import torch
    if kind == "relu":
        return v.clamp(min=0)
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    if kind == "gelu":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def linear_ref(x, w, wg=None, b=None, bg=None, r=None, act="none", out_bits=24):
    """-> (out, tol) in fp64.  tol: the fp32 product of K terms is off by at
    most (1.25 K + 32) half units (2^-24) of the sum of the terms' sizes
    (16 products a step, each and the running sum cut to 24 bits or more, the
    parts of a split reduction added after); the activations' slopes are at
    most 1.13 and their own error at most 16 half units of the value and 4 of
    the argument; then a product, a sum and the final rounding (out_bits: 24
    for fp32, 8 for bf16), half a unit each."""
    import torch
    u = 2.0 ** -24
    K = x.shape[1]

    def product(w, b):
        s = (x.double().abs() @ w.double().abs().T) + (0 if b is None else b.double().abs())
        v = x.double() @ w.double().T + (0 if b is None else b.double())
        return v, (1.25 * K + 32) * u * s

    v, ev = product(w, b)
    if wg is None:
        o = act64(v, act)
        e = ev if act == "none" else 1.13 * ev + 16 * u * o.abs() + 4 * u * v.abs()
    else:
        g, eg = product(wg, bg)
        a = act64(g, act)
        ea = eg if act == "none" else 1.13 * eg + 16 * u * a.abs() + 4 * u * g.abs()
        o = a * v
        e = ea * (v.abs() + ev) + a.abs() * ev + u * o.abs()
    if r is not None:
        o = o + r.double()
        e = e + u * o.abs()
    half = 2.0 ** -24 if out_bits == 24 else 2.0 ** -8
    return o, e + half * (o.abs() + e) + 2.0 ** -126


def linear_norm_tol(K, out_bits=24):
    """Relative 2-norm of the error: each of the K / 16 steps cuts the running
    sum by at most one unit (2^-23), all in one direction; the final rounding
    by at most half a unit; a gated output has two such factors."""
    import torch  # noqa: F401
    return 2 * ((K / 16 + 32) * 2.0 ** -23) + (2.0 ** -8 if out_bits == 8 else 2.0 ** -24)
