"""Cases of the routing, dense product and routed-layer operators: the inputs,
a plain statement of each operator in elementary torch operations, its
definition in 64 bits, and the calls of the library.

Operators:
  gate    logits -> experts and weights of every token
  linear  out = act(x W^T + b) + r, or act(x Wg^T + bg) * (x W^T + b) + r
  routed  the MXFP4 expert layer under a given routing
Sizes are the K3 layer's (hidden 7168, expert and shared hidden 1536, 896
experts, 16 picks) where they are not generic.
"""
import math

import numpy as np
import torch

own = False

D, FF, E, K = 7168, 1536, 896, 16


# ---------------------------------------------------------------- the cases --
def gate(name, T, experts, k, score, bias=False, groups=1, kept=1, group_top=1, renorm=False, scale=1.0, bf16=False):
    return {"name": name, "op": "gate", "T": T, "experts": experts, "k": k, "score": score, "bias": bias,
            "groups": groups, "kept": kept, "group_top": group_top, "renorm": renorm, "scale": scale, "bf16": bf16}


def linear(name, T, n, k, gated=False, act="none", bias=False, residual=False, fp32=False):
    return {"name": name, "op": "linear", "T": T, "n": n, "k": k, "gated": gated, "act": act, "bias": bias,
            "residual": residual, "fp32": fp32}


def routed(name, T, d, ff, experts, k, shared, missing=0.0):
    return {"name": name, "op": "routed", "T": T, "d": d, "ff": ff, "experts": experts, "k": k, "shared": shared,
            "missing": missing}


def listed():
    return [
        # one decode token's routing
        gate("gate_1_token", 1, E, K, "softmax"),
        # a decode batch of a model with 256 experts in 8 groups, logits straight from a bf16 product
        gate("gate_64_groups", 64, 256, 8, "sigmoid", bias=True, groups=8, kept=4, group_top=2, renorm=True, scale=2.5,
             bf16=True),
        # a long prompt: softmax weights as the layer's own router gives them
        gate("gate_4096_softmax", 4096, E, K, "softmax", renorm=True),
        # the largest prefill pass, one token short of it: sigmoid scores with a balance bias
        gate("gate_8191_sigmoid", 8191, E, K, "sigmoid", bias=True, renorm=True, scale=2.5),
        # one token's router product: fp32 logits
        linear("linear_1_router", 1, E, D, fp32=True),
        # a decode batch's down projection, added to the residual stream
        linear("linear_8_down", 8, D, FF, residual=True),
        # a short prompt through a gated feed-forward block's first product
        linear("linear_100_glu", 100, FF, D, gated=True, act="silu"),
        # odd and ragged everywhere: bias and GELU
        linear("linear_333_ragged", 333, 1001, 1000, act="gelu", bias=True),
        # a long prompt: gated first product and the projection back
        linear("linear_4096_glu", 4096, FF, D, gated=True, act="silu"),
        linear("linear_4095_down", 4095, D, FF, residual=True),
        # one decode token through the 16 experts that another router picked
        routed("routed_1_token", 1, D, FF, 64, K, FF),
        # a prompt's tokens under a given routing, some picks dropped by a capacity limit
        routed("routed_512_tokens", 512, D, FF, 64, K, FF, missing=0.05),
    ]


def logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "gate", "linear", "linear", "linear", "routed"])
    if op == "gate":
        groups = rng.choice([1, 1, 2, 4, 8, 7])
        size = logint(rng, max(2, 8 // groups), 1024 // groups)
        experts = groups * size
        kept = rng.randint(1, groups)
        k = min(rng.randint(1, 32), kept * size)
        c = gate("", logint(rng, 1, 8192), experts, k, rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                 groups=groups, kept=kept, group_top=rng.choice([1, 2]) if groups > 1 else 1,
                 renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), bf16=rng.random() < 0.3)
    elif op == "linear":
        gated = rng.random() < 0.4
        while True:
            T, n, k = logint(rng, 1, 4096), logint(rng, 64, D), 8 * logint(rng, 8, D // 8)
            if T * n * k * (2 if gated else 1) <= 4096 * FF * D * 2:
                break
        c = linear("", T, n, k, gated=gated, act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                   bias=rng.random() < 0.5, residual=rng.random() < 0.5, fp32=rng.random() < 0.25)
    else:
        experts = rng.randint(4, 64)
        k = rng.randint(1, min(16, experts))
        c = routed("", logint(rng, 1, 512), 64 * logint(rng, 4, D // 64), 64 * logint(rng, 2, FF // 64), experts, k,
                   rng.choice([0, 64 * logint(rng, 2, FF // 64)]), missing=rng.choice([0.0, 0.05]))
    del c["name"]
    return c


def work(case):
    c, T = case, case["T"]
    if c["op"] == "gate":
        n = T * c["experts"]
        return {"bytes": n * (2 if c["bf16"] else 4) + T * c["k"] * 8 + c["experts"] * 4 * c["bias"], "flops": 10 * n}
    if c["op"] == "linear":
        m, o = (2 if c["gated"] else 1), (4 if c["fp32"] else 2)
        return {"bytes": 2 * c["k"] * (T + m * c["n"]) + o * T * c["n"] * (2 if c["residual"] else 1)
                + 4 * m * c["n"] * c["bias"], "flops": 2 * T * c["n"] * c["k"] * m}
    pairs = T * c["k"] * (1 - c["missing"])
    # experts that at least one of the T tokens picked, each token picking k of them at random
    distinct = c["experts"] * (1 - (1 - c["k"] * (1 - c["missing"]) / c["experts"]) ** T)
    return {"bytes": distinct * 3 * c["d"] * c["ff"] * 17 / 32 + 6 * c["d"] * c["shared"] + 4 * T * c["d"]
            + 8 * T * c["k"], "flops": 6 * c["d"] * (pairs * c["ff"] + T * c["shared"])}


# --------------------------------------------------------------- the inputs --
def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    c, g, T = case, generator(seed), case["T"]
    bf = torch.bfloat16
    if c["op"] == "gate":
        # logits of a trained router: spread about 1.5, with some experts liked more by every token
        l = normal(g, T, c["experts"], std=1.5) + normal(g, 1, c["experts"], std=0.5)
        return {"logits": l.to(bf) if c["bf16"] else l,
                "bias": normal(g, c["experts"], std=0.05) if c["bias"] else None}
    if c["op"] == "linear":
        n, k = c["n"], c["k"]
        return {"x": normal(g, T, k, dtype=bf), "w": normal(g, n, k, std=k ** -0.5, dtype=bf),
                "wg": normal(g, n, k, std=k ** -0.5, dtype=bf) if c["gated"] else None,
                "b": normal(g, n, std=0.1) if c["bias"] else None,
                "bg": normal(g, n, std=0.1) if c["bias"] and c["gated"] else None,
                "r": normal(g, T, n, dtype=torch.float32 if c["fp32"] else bf) if c["residual"] else None}
    d, ff, n, k, fs = c["d"], c["ff"], c["experts"], c["k"], c["shared"]
    blobs = torch.randint(0, 256, (n, 3 * d * ff * 17 // 32), generator=g, device="cuda", dtype=torch.uint8)
    for m in range(3):  # the scale planes: exponents 118..124
        a = (m * 17 + 16) * d * ff // 32
        blobs[:, a:a + d * ff // 32] = torch.randint(118, 125, (n, d * ff // 32), generator=g, device="cuda",
                                                     dtype=torch.uint8)
    idx = torch.rand(T, n, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
    wt = torch.rand(T, k, generator=g, device="cuda") + 0.05
    wt = wt / wt.sum(1, keepdim=True)
    gone = torch.rand(T, k, generator=g, device="cuda") < c["missing"]
    return {"x": normal(g, T, d, dtype=bf), "blobs": blobs, "idx": torch.where(gone, -1, idx),
            "weight": torch.where(gone, 0.0, wt),
            "sg": normal(g, fs, d, std=0.16, dtype=bf) if fs else None,
            "su": normal(g, fs, d, std=0.16, dtype=bf) if fs else None,
            "sd": normal(g, d, fs, std=0.16, dtype=bf) if fs else None}


def prepare(case, seed):
    """Inputs and what a user's program keeps: descriptors, workspace, outputs."""
    c, T = case, case["T"]
    s = {"c": dict(case), **inputs(case, seed)}
    if own:
        import mxfp4_routed_expert_softmax_b200 as k3
        s["k3"] = k3
        if c["op"] == "gate":
            s["desc"] = k3.make_gate(c["experts"], c["k"],
                                     k3.K3MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else k3.K3MOE_SCORE_SOFTMAX,
                                     c["groups"], c["kept"], c["group_top"], c["scale"],
                                     (k3.K3MOE_RENORM_TOPK if c["renorm"] else 0)
                                     | (k3.K3MOE_LOGITS_BF16 if c["bf16"] else 0))
            s["oi"] = torch.empty(T, c["k"], dtype=torch.int32, device="cuda")
            s["ow"] = torch.empty(T, c["k"], dtype=torch.float32, device="cuda")
        elif c["op"] == "linear":
            act = {"none": k3.K3MOE_ACT_NONE, "relu": k3.K3MOE_ACT_RELU, "silu": k3.K3MOE_ACT_SILU,
                   "gelu": k3.K3MOE_ACT_GELU, "gelu_tanh": k3.K3MOE_ACT_GELU_TANH}[c["act"]]
            s["desc"] = k3.make_linear(c["n"], c["k"], act, k3.K3MOE_OUT_FP32 if c["fp32"] else 0)
            s["ws"] = k3.new_linear_workspace(s["desc"], T)
            s["out"] = torch.empty(T, c["n"], dtype=torch.float32 if c["fp32"] else torch.bfloat16, device="cuda")
        else:
            s["desc"] = k3.make_dims(c["d"], c["ff"], c["experts"], c["k"], c["shared"])
            s["ws"] = k3.new_workspace(s["desc"], T)
            nb = s["blobs"].shape[1]
            s["ptrs"] = torch.arange(c["experts"], dtype=torch.int64, device="cuda") * nb + s["blobs"].data_ptr()
            s["out"] = torch.empty(T, c["d"], dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- the calls --
def run(s):
    c = s["c"]
    if own:
        k3 = s["k3"]
        if c["op"] == "gate":
            k3.check(k3.k3moe_gate(s["logits"], c["T"], s["bias"], s["desc"], s["oi"], s["ow"]))
            return s["oi"], s["ow"]
        if c["op"] == "linear":
            k3.check(k3.k3moe_linear(s["x"], c["T"], s["w"], s["wg"], s["b"], s["bg"], s["r"], s["desc"], s["out"],
                                     s["ws"]))
            return s["out"]
        k3.check(k3.k3moe_layer_routed(s["x"], c["T"], s["idx"], s["weight"], s["ptrs"], s["sg"], s["su"], s["sd"],
                                       s["desc"], s["out"], s["ws"]))
        return s["out"]
    return {"gate": plain_gate, "linear": plain_linear, "routed": plain_routed}[c["op"]](s)


def plain_gate(s):
    # 64 bits: scores next to one another decide which experts are picked
    c, l, n = s["c"], s["logits"].double(), s["c"]["experts"]
    none = -math.inf
    out = ~(l > none)
    if c["score"] == "softmax":
        m = l.masked_fill(out, none).amax(1, keepdim=True)
        e = torch.exp(l - torch.where(m > none, m, 0.0))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    # without a bias the order of the scores is the order of the logits
    c_score = score + s["bias"].double() if c["bias"] else score
    order = c_score if c["bias"] else l
    out = out | ~(order > none)
    order = order.masked_fill(out, none)
    if c["groups"] > 1:
        per = (order if c["group_top"] == 1 else c_score.masked_fill(out, none)).view(-1, c["groups"], n // c["groups"])
        group = per.sort(dim=2, descending=True)[0][..., :c["group_top"]].sum(2)
        kept = group.sort(dim=1, descending=True, stable=True)[1][:, :c["kept"]]
        keep = torch.zeros_like(group, dtype=torch.bool).scatter_(1, kept, True)
        order = order.masked_fill(~keep.repeat_interleave(n // c["groups"], 1), none)
    top, idx = (v[:, :c["k"]] for v in order.sort(dim=1, descending=True, stable=True))
    w = score.gather(1, idx).masked_fill(top == none, 0.0)
    if c["renorm"]:
        z = w.sum(1, keepdim=True)
        w = torch.where(z == 0.0, 0.0, w / z)
    return idx.masked_fill(top == none, -1).to(torch.int32), (w * c["scale"]).float()


def activation(v, kind):
    if kind == "relu":
        return torch.maximum(v, torch.zeros_like(v))
    if kind == "silu":
        return v / (1.0 + torch.exp(-v))
    if kind == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * 0.5 ** 0.5))
    if kind == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))
    return v


def plain_linear(s):
    c, x = s["c"], s["x"].float()

    def product(w, b):
        v = x @ w.float().T
        return v if b is None else v + b

    v = product(s["w"], s["b"])
    v = activation(product(s["wg"], s["bg"]), c["act"]) * v if c["gated"] else activation(v, c["act"])
    if s["r"] is not None:
        v = v + s["r"].float()
    return v if c["fp32"] else v.to(torch.bfloat16)


def unpack(blobs, m, rows, cols):
    """Matrix m of every expert blob given, [experts, rows, cols] in 32 bits."""
    a = m * rows * cols * 17 // 32
    nib = blobs[:, a:a + rows * cols // 2]
    sc = blobs[:, a + rows * cols // 2:a + rows * cols * 17 // 32]
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=blobs.device)
    codes = torch.stack((nib & 15, nib >> 4), 2).view(-1, rows * cols // 32, 32)
    return (table[codes.int()] * torch.exp2(sc.float() - 127.0)[..., None]).view(-1, rows, cols)


def plain_routed(s):
    c, x, idx = s["c"], s["x"].float(), s["idx"].long()
    T, d, ff, n, k = c["T"], c["d"], c["ff"], c["experts"], c["k"]
    # the picked experts, and each pick's place among its expert's tokens
    hit = torch.nn.functional.one_hot(idx + 1, n + 1)[..., 1:].sum(1)  # [T, n]
    used = hit.any(0).nonzero()[:, 0]
    place = hit.cumsum(0) - hit
    room = max(1, int(hit.sum(0).max()))
    slot = torch.zeros(n, dtype=torch.long, device="cuda").index_copy(0, used, torch.arange(len(used), device="cuda"))
    there = idx >= 0
    at = slot[idx.clamp(min=0)] * room + place.gather(1, idx.clamp(min=0))  # [T, k]
    xs = torch.zeros(len(used) * room, d, device="cuda")
    token = torch.arange(T, device="cuda")[:, None].expand(T, k)
    xs[at[there]] = x[token[there]]
    xs, blobs = xs.view(len(used), room, d), s["blobs"][used]
    h = activation(xs @ unpack(blobs, 0, ff, d).transpose(1, 2), "silu") * (xs @ unpack(blobs, 1, ff, d).transpose(1, 2))
    o = (h @ unpack(blobs, 2, d, ff).transpose(1, 2)).view(-1, d)
    y = torch.zeros(T, d, device="cuda")
    if len(used):
        y = (o[at] * (s["weight"] * there)[..., None]).sum(1)
    if c["shared"]:
        y = y + (activation(x @ s["sg"].float().T, "silu") * (x @ s["su"].float().T)) @ s["sd"].float().T
    return y.to(torch.bfloat16)


# ------------------------------------------------ the definition in 64 bits --
def exact(case, seed):
    c, s, T = case, inputs(case, seed), case["T"]
    if c["op"] == "gate":
        return exact_gate(c, s["logits"].float().cpu().numpy().astype(np.float64),
                          None if s["bias"] is None else s["bias"].cpu().numpy().astype(np.float64))
    f64 = {a: v.double() for a, v in s.items() if v is not None and v.is_floating_point()}

    def act(v, kind):
        if kind == "relu":
            return v.clamp(min=0)
        if kind == "silu":
            return v * torch.sigmoid(v)
        if kind == "gelu":
            return v * torch.special.ndtr(v)
        if kind == "gelu_tanh":
            return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
        return v

    if c["op"] == "linear":
        v = torch.nn.functional.linear(f64["x"], f64["w"], f64.get("b"))
        v = act(torch.nn.functional.linear(f64["x"], f64["wg"], f64.get("bg")), c["act"]) * v if c["gated"] else act(v, c["act"])
        return v + f64["r"] if "r" in f64 else v
    d, ff, x = c["d"], c["ff"], f64["x"]

    def matrix(blob, m, rows, cols):
        mat = blob[m * rows * cols * 17 // 32:(m + 1) * rows * cols * 17 // 32]
        b = mat[:rows * cols // 2].view(rows, cols // 2).int()
        v = torch.empty(rows, cols, dtype=torch.float64, device=blob.device)
        for half in range(2):
            code = (b >> (4 * half)) & 15
            e, f = (code >> 1) & 3, (code & 1).double()
            mag = torch.where(e > 0, torch.ldexp(1.0 + f / 2, e - 1), f / 2)
            v[:, half::2] = torch.where(code >= 8, -mag, mag)
        sc = mat[rows * cols // 2:].view(rows, cols // 32).int() - 127
        return torch.ldexp(v.view(rows, cols // 32, 32), sc[..., None]).view(rows, cols)

    y = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        t, j = (s["idx"] == e).nonzero(as_tuple=True)
        if len(t):
            xe, blob = x[t], s["blobs"][e]
            h = act(xe @ matrix(blob, 0, ff, d).T, "silu") * (xe @ matrix(blob, 1, ff, d).T)
            y.index_add_(0, t, (h @ matrix(blob, 2, d, ff).T) * f64["weight"][t, j, None])
    if c["shared"]:
        y += (act(x @ f64["sg"].T, "silu") * (x @ f64["su"].T)) @ f64["sd"].T
    return y


def exact_gate(c, l, bias):
    n, g, k = c["experts"], c["groups"], c["k"]
    idx, w = np.full((len(l), k), -1, np.int32), np.zeros((len(l), k))
    for t, row in enumerate(l):
        with np.errstate(over="ignore", invalid="ignore"):
            score = 1 / (1 + np.exp(-row)) if c["score"] == "sigmoid" else np.exp(row - row.max())
            score = score if c["score"] == "sigmoid" else score / score.sum()
        value = score if bias is None else score + bias
        order = row if bias is None else value
        left = np.nonzero(order > -np.inf)[0]
        left = left[row[left] > -np.inf]
        if g > 1:
            total = np.full(g, -np.inf)
            for q in range(g):
                mine = np.sort(value[left[left // (n // g) == q]])[::-1]
                if len(mine) >= c["group_top"]:
                    total[q] = mine[:c["group_top"]].sum()
            kept = np.lexsort((np.arange(g), -total))[:c["kept"]]
            left = left[np.isin(left // (n // g), kept)]
        pick = left[np.lexsort((left, -order[left]))][:k]
        z = score[pick].sum() if c["renorm"] else 1.0
        idx[t, :len(pick)] = pick
        w[t, :len(pick)] = c["scale"] * score[pick] / z if z else 0.0
    return idx, w
