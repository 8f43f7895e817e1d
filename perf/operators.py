"""The cases by which the training operators of the routed adapters are measured.

Three operators, as a training step of token-routed LoRA adapters uses them:

  route   experts for every token from router logits: softmax or sigmoid scores, a selection bias,
          groups, top k, renormalised weights; with its gradient
  sgmmb   the gradients of the batched adapter product y += s sum_k g_k (x A_k^T) B_k^T
  adamw   one AdamW step over many tensors, with moments in 32 or in 8 bits

A case is a dict of plain values; prepare() makes its inputs on the GPU from a seed, run() does one
pass: the plain form (elementary torch operations) or, with own set, the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}

# One decoder layer of the 7B-shaped workload: (d_out, d_in) of its seven adapted projections.
LAYER_7B = [(4096, 4096)] * 4 + [(11008, 4096)] * 2 + [(4096, 11008)]


def listed():
    return [
        # a decode batch: 64 rows, top 2 of 8 adapters; latency is all there is
        {"name": "route-decode", "op": "route", "T": 64, "E": 8, "k": 2, "score": "softmax", "bias": 0, "groups": 1,
         "keep": 1, "group_top": 1, "renorm": 1, "scale": 1.0, "dtype": "f32", "pad": 0, "masked": 0.0, "grad": 0},
        # a ragged batch with padding rows and unavailable experts, softmax weights kept as they are
        {"name": "route-ragged", "op": "route", "T": 4099, "E": 60, "k": 6, "score": "softmax", "bias": 0, "groups": 1,
         "keep": 1, "group_top": 1, "renorm": 0, "scale": 1.0, "dtype": "bf16", "pad": 131, "masked": 0.1, "grad": 1},
        # a large prefill batch over many small experts: sigmoid scores, balance bias, 4 of 8 groups, top 8
        {"name": "route-prefill", "op": "route", "T": 32768, "E": 256, "k": 8, "score": "sigmoid", "bias": 1, "groups": 8,
         "keep": 4, "group_top": 2, "renorm": 1, "scale": 2.5, "dtype": "f32", "pad": 0, "masked": 0.0, "grad": 0},
        # the training step's router: the same routing with the gradient of its weights
        {"name": "route-train", "op": "route", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": 1, "groups": 8,
         "keep": 4, "group_top": 2, "renorm": 1, "scale": 2.5, "dtype": "bf16", "pad": 0, "masked": 0.0, "grad": 1},
        # a short fine-tuning batch through one projection
        {"name": "sgmmb-short", "op": "sgmmb", "T": 256, "shape": "4096x4096", "n": 1, "E": 8, "r": 16, "zipf": 1.1,
         "dtype": "bf16", "pad": 0},
        # odd sizes in single precision, with padding rows behind the last sequence
        {"name": "sgmmb-ragged-f32", "op": "sgmmb", "T": 523, "shape": "1000x776", "n": 2, "E": 4, "r": 4, "zipf": 0.0,
         "dtype": "f32", "pad": 37},
        # one 7B-shaped layer's seven projections at the prefill workload's 4096 tokens
        {"name": "sgmmb-layer", "op": "sgmmb", "T": 4096, "shape": "7b", "n": 1, "E": 8, "r": 16, "zipf": 1.1,
         "dtype": "bf16", "pad": 0},
        # a 70B-shaped projection: 16 adapters of rank 64
        {"name": "sgmmb-wide", "op": "sgmmb", "T": 4096, "shape": "8192x8192", "n": 1, "E": 16, "r": 64, "zipf": 1.1,
         "dtype": "bf16", "pad": 0},
        # one layer's adapter banks, 14 tensors: bf16 weights with fp32 masters
        {"name": "adamw-layer", "op": "adamw", "layers": 1, "E": 8, "r": 16, "odd": 0, "p": "bf16", "master": 1,
         "g": "f32", "bits": 32},
        # the same with 8-bit moments
        {"name": "adamw8-layer", "op": "adamw", "layers": 1, "E": 8, "r": 16, "odd": 0, "p": "bf16", "master": 1,
         "g": "f32", "bits": 8},
        # eight layers' banks of odd sizes, fp32 weights, 8-bit moments
        {"name": "adamw8-odd", "op": "adamw", "layers": 8, "E": 8, "r": 16, "odd": 1, "p": "f32", "master": 0,
         "g": "f32", "bits": 8},
        # every adapter of the 7B-shaped model: 448 tensors, 322 million weights
        {"name": "adamw-model", "op": "adamw", "layers": 32, "E": 8, "r": 16, "odd": 0, "p": "bf16", "master": 1,
         "g": "f32", "bits": 32},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "sgmmb", "adamw"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.randint(2, 32) if groups > 1 else rng.randint(2, 256)
        keep = rng.randint(1, groups)
        return {"op": "route", "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, keep * (E // groups))),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.randint(0, 1), "groups": groups, "keep": keep,
                "group_top": rng.choice([1, 2]), "renorm": rng.randint(0, 1), "scale": rng.choice([1.0, 2.5]),
                "dtype": rng.choice(["f32", "bf16"]), "pad": rng.choice([0, 5]), "masked": rng.choice([0.0, 0.1]),
                "grad": rng.randint(0, 1)}
    if op == "sgmmb":
        dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
        if dt == "f32":  # the element-wise path: small sizes
            return {"op": "sgmmb", "T": _log(rng, 1, 600), "shape": "%dx%d" % (_log(rng, 8, 1024), _log(rng, 8, 1024)),
                    "n": rng.randint(1, 3), "E": rng.randint(2, 8), "r": rng.randint(1, 8), "zipf": 1.1,
                    "dtype": dt, "pad": rng.choice([0, 7])}
        return {"op": "sgmmb", "T": _log(rng, 1, 4096), "shape": "%dx%d" % (8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 1024)),
                "n": rng.randint(1, 3), "E": rng.randint(2, 16), "r": rng.choice([4, 8, 16, 16, 24, 32, 64]),
                "zipf": rng.choice([0.0, 1.1]), "dtype": dt, "pad": rng.choice([0, 7])}
    return {"op": "adamw", "layers": _log(rng, 1, 16), "E": rng.choice([4, 8]), "r": rng.choice([4, 8, 16]),
            "odd": rng.randint(0, 1), "p": rng.choice(["f32", "bf16"]), "master": 1, "g": rng.choice(["f32", "bf16"]),
            "bits": rng.choice([32, 8])}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _shapes(c):
    if c["shape"] == "7b":
        return LAYER_7B * c["n"]
    o, i = (int(v) for v in c["shape"].split("x"))
    return [(o, i)] * c["n"]


def _sizes(c):
    """Element counts of the tensors of an adamw case: A [E][r][d_in] and B [E][d_out][r] of every projection."""
    n = [c["E"] * c["r"] * d for _ in range(c["layers"]) for o, i in LAYER_7B for d in (i, o)]
    return [v - 7 * j - 1 for j, v in enumerate(n)] if c["odd"] else n


BLOCK = 256  # elements of a block of 8-bit moments


def prepare(c, seed):
    return {"route": _prepare_route, "sgmmb": _prepare_sgmmb, "adamw": _prepare_adamw}[c["op"]](c, seed)


def run(s):
    return {"route": _run_route, "sgmmb": _run_sgmmb, "adamw": _run_adamw}[s["c"]["op"]](s)


def work(c):
    if c["op"] == "route":
        e, n = (4 if c["dtype"] == "f32" else 2), c["T"] * c["E"]
        b = n * e + c["T"] * c["k"] * 8 + (4 * c["E"] if c["bias"] else 0)
        if c["grad"]:
            b += c["T"] * c["k"] * 4 + n * e
        return {"bytes": b, "flops": 10 * n}
    if c["op"] == "sgmmb":
        e, T, E, r = (4 if c["dtype"] == "f32" else 2), c["T"], c["E"], c["r"]
        b = T * (2 * 8 + 2 * 4)
        f = 0
        for o, i in _shapes(c):
            b += e * (T * i + T * o + 2 * T * i) + E * r * (i + o) * (e + 4)  # x, dy, dx read and written; banks, their gradients
            f += 2 * T * 2 * r * (2 * o + 3 * i)
        return {"bytes": b, "flops": f}
    n = sum(_sizes(c))
    p, g = (4 if c["p"] == "f32" else 2), (4 if c["g"] == "f32" else 2)
    b = n * g + (n * (8 + p) if c["p"] == "bf16" and c["master"] else 2 * n * p)
    b += n * 16 if c["bits"] == 32 else n * (4 + 8) + n // BLOCK * 24  # 8 bits: the moments' values come back too
    return {"bytes": b, "flops": 16 * n}


# ------------------------------------------------------------------ routing

def _prepare_route(c, seed):
    g = _gen(seed)
    T, E = c["T"], c["E"]
    logits = torch.randn((T, E), generator=g, device=DEV) * 1.5
    if c["masked"]:
        off = torch.rand((T, E), generator=g, device=DEV) < c["masked"]
        logits = logits.masked_fill(off, -math.inf)
    if c["pad"]:
        logits[max(T - c["pad"], 1):] = -math.inf  # padding rows: no expert is available
    s = {"c": c, "logits": logits.to(DT[c["dtype"]]), "bias": None, "dg": None}
    if c["bias"]:
        s["bias"] = torch.randn(E, generator=g, device=DEV) * 0.05
    if c["grad"]:
        s["dg"] = torch.randn((T, c["k"]), generator=g, device=DEV)
    return s


def _run_route(s):
    c, logits = s["c"], s["logits"]
    if own:
        import dynamic_lora_moe_amd as dlm

        idx, g = dlm.route(logits, c["k"], score=c["score"], bias=s["bias"], n_groups=c["groups"], keep_groups=c["keep"],
                           group_top=c["group_top"], renorm=bool(c["renorm"]), scale=c["scale"])
        if not c["grad"]:
            return {"idx": idx, "g": g}
        return {"idx": idx, "g": g, "dlogits": dlm.route_backward(logits, idx, s["dg"], score=c["score"],
                                                                  renorm=bool(c["renorm"]), scale=c["scale"])}
    T, E = logits.shape
    l = logits.double()  # the order of scores next to one another decides: 64 bits
    live = l > -math.inf
    if c["score"] == "softmax":
        top = l.amax(1, keepdim=True).clamp(min=-1e300)
        p = torch.exp(l - top)
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        p = 1 / (1 + torch.exp(-l))
    key = p + s["bias"].double() if s["bias"] is not None else p
    key = torch.where(live, key, -math.inf)
    if c["groups"] > 1:
        kg = key.view(T, c["groups"], -1)
        best = kg.amax(2)
        if c["group_top"] == 2 and kg.shape[2] > 1:
            second = kg.scatter(2, kg.argmax(2, keepdim=True), -math.inf).amax(2)
            best = best + torch.where(second > -math.inf, second, 0.0)
        kept = torch.zeros_like(best, dtype=torch.bool)
        for _ in range(c["keep"]):
            a = best.argmax(1, keepdim=True)
            kept.scatter_(1, a, best.gather(1, a) > -math.inf)
            best = best.scatter(1, a, -math.inf)
        key = torch.where(kept[:, :, None], kg, -math.inf).reshape(T, E)
    picks = []
    for _ in range(c["k"]):
        a = key.argmax(1, keepdim=True)
        picks.append(torch.where(key.gather(1, a) > -math.inf, a, -1))
        key = key.scatter(1, a, -math.inf)
    idx = torch.cat(picks, 1)
    on, at = idx >= 0, idx.clamp(min=0)
    w = torch.where(on, p.gather(1, at), 0.0)
    if c["renorm"]:
        tot = w.sum(1, keepdim=True)
        q = torch.where(tot > 0, w / tot.clamp(min=1e-300), 0.0)
    else:
        tot, q = None, w
    out = {"idx": idx.int(), "g": (q * c["scale"]).float()}
    if not c["grad"]:
        return out
    d = torch.where(on, s["dg"].double(), 0.0) * c["scale"]
    if c["renorm"]:
        d = torch.where(tot > 0, (d - (d * q).sum(1, keepdim=True)) / tot.clamp(min=1e-300), 0.0)
    dp = torch.zeros_like(l).scatter_add_(1, at, torch.where(on, d, 0.0))
    if c["score"] == "softmax":
        dl = p * (dp - (dp * p).sum(1, keepdim=True))
    else:
        dl = dp * p * (1 - p)
    out["dlogits"] = torch.where(live, dl, 0.0).to(logits.dtype)
    return out


def _exact_route(c, seed):
    s = _prepare_route(c, seed)
    l, n = s["logits"].double(), c["E"] // c["groups"]
    dead = torch.isneginf(l)
    sc = torch.nan_to_num(torch.softmax(l, 1)) if c["score"] == "softmax" else torch.sigmoid(l)
    sel = sc if s["bias"] is None else sc + s["bias"].double()
    sel = sel.masked_fill(dead, -math.inf)
    if c["groups"] > 1:
        v = sel.view(c["T"], c["groups"], n).sort(dim=2, descending=True).values[:, :, :c["group_top"]]
        v = torch.where(v.isneginf(), torch.tensor(0.0, device=DEV, dtype=torch.float64), v).sum(2)
        v = v.masked_fill(dead.view(c["T"], c["groups"], n).all(2), -math.inf)
        order = v.sort(dim=1, descending=True, stable=True).indices[:, c["keep"]:]
        lost = torch.zeros_like(v, dtype=torch.bool).scatter_(1, order, True)
        sel = sel.masked_fill(lost.repeat_interleave(n, 1), -math.inf)
    top = sel.sort(dim=1, descending=True, stable=True)
    best, at = top.values[:, :c["k"]], top.indices[:, :c["k"]]
    hot = torch.zeros(c["T"], c["k"], c["E"], device=DEV, dtype=torch.float64).scatter_(2, at[:, :, None], 1.0)
    hot = hot * (~best.isneginf())[:, :, None]
    # the weights as a function of the scores, with autograd for the gradient
    z = l.masked_fill(dead, 0.0).requires_grad_(True)
    zz = z.masked_fill(dead, -math.inf)
    f = torch.where(dead.all(1, keepdim=True), 0.0, torch.softmax(torch.where(dead.all(1, keepdim=True), 0.0, zz), 1)) \
        if c["score"] == "softmax" else torch.where(dead, 0.0, torch.sigmoid(z))
    w = (hot * f[:, None, :]).sum(2)
    if c["renorm"]:
        t = w.sum(1, keepdim=True)
        w = w / torch.where(t > 0, t, 1.0)
    w = w * c["scale"]
    out = {"idx": None, "g": w.detach()}
    if c["grad"]:
        w.backward(s["dg"].double())
        out["dlogits"] = z.grad
    return out


# ------------------------------------------------------------------ the adapters' gradients

SCALE = 2.0


def _prepare_sgmmb(c, seed):
    g, dt = _gen(seed), DT[c["dtype"]]
    T, E, r = c["T"], c["E"], c["r"]
    w = (1.0 / torch.arange(1, E + 1, device=DEV) ** c["zipf"]).expand(T, E)
    idx = torch.multinomial(w, 2, generator=g).int()
    gate = torch.softmax(torch.randn((T, 2), generator=g, device=DEV), 1)
    if c["pad"]:
        idx[max(T - c["pad"], 1):] = -1  # padding rows: both slots empty
        if T >= 16:
            idx[0, 1] = -1  # a row with one expert
    rnd = lambda std, *shape: (torch.randn(shape, generator=g, device=DEV) * std).to(dt)  # noqa: E731
    s = {"c": c, "idx": idx, "g": gate, "x": [], "A": [], "B": [], "dy": [], "dx": [], "y": []}
    for o, i in _shapes(c):
        s["x"].append(rnd(1.0, T, i))
        s["A"].append(rnd(0.02, E, r, i))
        s["B"].append(rnd(0.02, E, o, r))
        s["dy"].append(rnd(1.0, T, o))
        s["dx"].append(rnd(1.0, T, i))  # the base product's gradient, which the adapters' joins
    # what the step keeps: the gradients' buffers
    s["dA"] = [torch.empty(A.shape, device=DEV) for A in s["A"]]
    s["dB"] = [torch.empty(B.shape, device=DEV) for B in s["B"]]
    s["dg"] = torch.empty((T, 2), device=DEV)
    if own:
        import dynamic_lora_moe_amd as dlm

        s["y"] = [torch.zeros_like(d) for d in s["dy"]]
        s["grp"] = dlm.SgmmGroup(list(zip(s["x"], s["A"], s["B"], s["y"])), E, r, SCALE)
        s["grp"].bind_grads(s["dy"], s["dx"], s["dA"], s["dB"])
        s["ws"] = s["grp"].backward_workspace(T)
    return s


def _run_sgmmb(s):
    if own:
        s["grp"].backward(s["idx"], s["g"], s["dg"], workspace=s["ws"])
        return {"dx": s["dx"], "dA": s["dA"], "dB": s["dB"], "dg": s["dg"]}
    T, E, r = s["c"]["T"], s["c"]["E"], s["c"]["r"]
    at = s["idx"].long().clamp(min=0)
    on = (s["idx"] >= 0).float()
    # every token's gate of every expert, and which expert each slot has
    hot = torch.zeros((T, 2, E), device=DEV).scatter_(2, at[:, :, None], on[:, :, None])
    gate = SCALE * (hot * s["g"][:, :, None]).sum(1)
    dg = 0.0
    for p in range(len(s["x"])):
        x, dy = s["x"][p].float(), s["dy"][p].float()
        A, B = s["A"][p].float().view(E * r, -1), s["B"][p].float()
        B = B.transpose(1, 2).reshape(E * r, -1)
        u = (x @ A.t()).view(T, E, r)
        w = (dy @ B.t()).view(T, E, r)
        dg = dg + SCALE * (hot * (u * w).sum(2)[:, None, :]).sum(2)
        gw, gu = (gate[:, :, None] * w).view(T, E * r), (gate[:, :, None] * u).view(T, E * r)
        s["dx"][p].copy_(s["dx"][p].float() + gw @ A)
        s["dA"][p].copy_((gw.t() @ x).view(E, r, -1))
        s["dB"][p].copy_((dy.t() @ gu).view(-1, E, r).transpose(0, 1))
    s["dg"].copy_(dg)
    return {"dx": s["dx"], "dA": s["dA"], "dB": s["dB"], "dg": s["dg"]}


def _exact_sgmmb(c, seed):
    global own
    was, own = own, False
    s = _prepare_sgmmb(c, seed)
    own = was
    T, E = c["T"], c["E"]
    out = {"dx": [], "dA": [], "dB": [], "dg": torch.zeros((T, 2), device=DEV, dtype=torch.float64)}
    rows = [[(s["idx"][:, k] == e).nonzero().flatten() for k in (0, 1)] for e in range(E)]
    g = s["g"].double() * SCALE
    for x, A, B, dy, dx in zip(s["x"], s["A"], s["B"], s["dy"], s["dx"]):
        x, A, B, dy, dx = (v.double() for v in (x, A, B, dy, dx))
        dA, dB = torch.zeros_like(A), torch.zeros_like(B)
        for e in range(E):
            for k in (0, 1):
                t = rows[e][k]
                u, w = x[t] @ A[e].t(), dy[t] @ B[e]
                out["dg"][t, k] += SCALE * (u * w).sum(1)
                u, w = u * g[t, k, None], w * g[t, k, None]
                dx[t] += w @ A[e]
                dA[e] += w.t() @ x[t]
                dB[e] += dy[t].t() @ u
        out["dx"].append(dx)
        out["dA"].append(dA)
        out["dB"].append(dB)
    return out


# ------------------------------------------------------------------ AdamW

LR, B1, B2, EPS, WD, STEP0, SEED = 1e-3, 0.9, 0.999, 1e-8, 0.01, 10, 20260312


def _prepare_adamw(c, seed):
    gen = _gen(seed)
    sizes = _sizes(c)
    blocks = [-(-n // BLOCK) for n in sizes]
    n = sum(blocks) * BLOCK
    first = [0]
    for b in blocks:
        first.append(first[-1] + b * BLOCK)
    # every tensor starts at a whole block of one flat buffer; what lies behind its end is zero and stays so
    live = torch.zeros(n, dtype=torch.bool, device=DEV)
    for f, k in zip(first, sizes):
        live[f:f + k] = True
    w = torch.randn(n, generator=gen, device=DEV) * 0.02 * live
    s = {"c": c, "lr": LR, "live": live if c["odd"] else None, "step": STEP0, "sizes": sizes, "first": first}
    s["p"] = w.to(DT[c["p"]])
    s["master"] = w if c["master"] and c["p"] == "bf16" else None
    s["g"] = (torch.randn(n, generator=gen, device=DEV) * 1e-3 * live).to(DT[c["g"]])
    if c["bits"] == 32:
        s["m"] = torch.randn(n, generator=gen, device=DEV) * 3e-4 * live
        s["v"] = (torch.rand(n, generator=gen, device=DEV) + 0.1) * 1e-6 * live
    else:
        s["m"] = (torch.randint(-127, 128, (n,), generator=gen, device=DEV) * live).to(torch.int8)
        s["v"] = (torch.randint(90, 256, (n,), generator=gen, device=DEV) * live).to(torch.uint8)
        s["ms"] = (torch.rand(sum(blocks), generator=gen, device=DEV) + 0.5) * 1e-3
        s["vs"] = (torch.rand(sum(blocks), generator=gen, device=DEV) + 0.5) * 4e-6
        t = torch.arange(len(sizes), device=DEV)
        per = torch.tensor(blocks, device=DEV)
        s["tensor"] = t.repeat_interleave(per)
        s["block"] = torch.arange(sum(blocks), device=DEV) - (per.cumsum(0) - per).repeat_interleave(per)
    if own:
        import dynamic_lora_moe_amd as dlm

        cut = lambda v: None if v is None else [v[f:f + k] for f, k in zip(first, sizes)]  # noqa: E731
        cutb = lambda v: [v[f // BLOCK:f // BLOCK + b] for f, b in zip(first, blocks)]  # noqa: E731
        state = list(zip(cut(s["m"]), cut(s["v"]))) if c["bits"] == 32 else \
            list(zip(cut(s["m"]), cut(s["v"]), cutb(s["ms"]), cutb(s["vs"])))
        s["opt"] = dlm.AdamW(cut(s["p"]), cut(s["g"]), masters=cut(s["master"]), state_bits=c["bits"], states=state,
                             beta1=B1, beta2=B2, eps=EPS, weight_decay=WD, step=STEP0, seed=SEED)
    return s


M32 = 0xFFFFFFFF


def _mix(x):
    """The 32-bit finaliser of MurmurHash3 (A. Appleby, public domain) on values held in 64 bits."""
    x = (x ^ (x >> 16)) * 0x85EBCA6B & M32
    x = (x ^ (x >> 13)) * 0xC2B2AE35 & M32
    return x ^ (x >> 16)


def _noise(s):
    """Two numbers of 16 bits for every element, as fractions in (0, 1): functions of seed, step, tensor, block and place."""
    key = _mix(torch.tensor((SEED & M32) + s["step"] * 0x9E3779B1 & M32, device=DEV))
    key = _mix((key + s["tensor"] * 0x85EBCA77) & M32)
    key = _mix((key + s["block"] * 0xC2B2AE3D) & M32)
    h = _mix((key[:, None] + torch.arange(BLOCK, device=DEV) * 0x9E3779B1) & M32)
    return ((h & 0xFFFF).double() + 0.5) / 65536, ((h >> 16).double() + 0.5) / 65536


def _run_adamw(s):
    c = s["c"]
    if own:
        import dynamic_lora_moe_amd as dlm

        s["opt"].step(s["lr"])
        out = {"p": s["p"]}
        if s["master"] is not None:
            out["master"] = s["master"]
        if c["bits"] == 32:
            return out | {"m": s["m"], "v": s["v"]}
        m, v = dlm.adamw_read_state(s["m"], s["v"], s["ms"], s["vs"])
        return out | {"m": m, "v": v}
    s["step"] += 1
    c1, c2 = 1 - B1 ** s["step"], 1 - B2 ** s["step"]
    g = s["g"].float()
    if c["bits"] == 32:
        m, v = s["m"].mul_(B1).add_(g, alpha=1 - B1), s["v"].mul_(B2).add_(g * g, alpha=1 - B2)
    else:  # the codes turn on values next to a border: 64 bits
        q, k = s["m"].double().view(-1, BLOCK), s["v"].double().view(-1, BLOCK)
        gd = g.double().view(-1, BLOCK)
        m = B1 * (s["ms"].double()[:, None] * (q * q.abs() / 127 ** 2)) + (1 - B1) * gd
        v = B2 * (s["vs"].double()[:, None] * ((k * k) * (k * k) / 255 ** 4)) + (1 - B2) * (gd * gd)
        um, uv = _noise(s)
        ms, vs = m.abs().amax(1).float(), v.amax(1).float()
        x = torch.where(ms[:, None] > 0, m.abs() * (127 ** 2 / ms.double()[:, None]), 0.0).clamp(max=127.0 ** 2)
        lo = torch.floor(torch.sqrt(x))
        lo = (lo + (x - lo * lo > um * (2 * lo + 1))) * torch.sign(m)
        x = torch.where(vs[:, None] > 0, v * (255 ** 4 / vs.double()[:, None]), 0.0).clamp(max=255.0 ** 4)
        b = torch.floor(torch.sqrt(torch.sqrt(x)))
        b4, b5 = b ** 4, (b + 1) ** 4
        b = b + (x - b4 > uv * (b5 - b4))
        b = torch.where((v > 0) & (vs[:, None] > 0), b.clamp(min=1), b)
        s["m"].copy_(lo.view(-1))
        s["v"].copy_(b.view(-1))
        s["ms"].copy_(ms)
        s["vs"].copy_(vs)
        qm = (ms.double()[:, None] * (lo * lo.abs() / 127 ** 2)).view(-1).float()
        qv = (vs.double()[:, None] * ((b * b) * (b * b) / 255 ** 4)).view(-1).float()
        m, v = m.view(-1).float(), v.view(-1).float()
    w = s["master"] if s["master"] is not None else s["p"].float()
    w = w * (1 - LR * WD) - LR * ((m / c1) / (torch.sqrt(v / c2) + EPS))
    s["p"].copy_(w)
    out = {"p": s["p"]}
    if s["master"] is not None:
        s["master"].copy_(w)
        out["master"] = s["master"]
    return out | ({"m": m, "v": v} if c["bits"] == 32 else {"m": qm, "v": qv})


def _exact_adamw(c, seed):
    global own
    was, own = own, False
    s = _prepare_adamw(c, seed)
    own = was
    t = STEP0 + 1
    names = ["p", "m", "v"] + (["master"] if s["master"] is not None else [])
    out = {k: torch.zeros(s["p"].numel(), dtype=torch.float32 if s["p"].numel() > 1 << 27 else torch.float64, device=DEV)
           for k in names}
    u32 = lambda x: x % 4294967296  # noqa: E731

    def final(h):
        h = u32((h ^ torch.div(h, 65536, rounding_mode="floor")) * 2246822507)
        h = u32((h ^ torch.div(h, 8192, rounding_mode="floor")) * 3266489909)
        return h ^ torch.div(h, 65536, rounding_mode="floor")

    for j, (f, n) in enumerate(zip(s["first"], s["sizes"])):
        cut = slice(f, f + n)
        g = s["g"][cut].double()
        if c["bits"] == 32:
            m, v = s["m"][cut].double(), s["v"][cut].double()
        else:
            nb = -(-n // BLOCK)
            b0 = f // BLOCK
            own_block = torch.div(torch.arange(n, device=DEV), BLOCK, rounding_mode="floor")
            a, b = s["m"][cut].double() / 127, s["v"][cut].double() / 255
            m = s["ms"][b0:b0 + nb].double()[own_block] * torch.sign(a) * a.square()
            v = s["vs"][b0:b0 + nb].double()[own_block] * b.square().square()
        m = m * B1 + g * (1 - B1)
        v = v * B2 + g.square() * (1 - B2)
        w = (s["master"] if s["master"] is not None else s["p"])[cut].double()
        w = w - LR * WD * w - LR * (m / (1 - B1 ** t)) / ((v / (1 - B2 ** t)).sqrt() + EPS)
        if c["bits"] == 8:
            h = final(torch.full((1,), u32(SEED + t * 2654435761), device=DEV))
            h = final(u32(h + j * 2246822519))
            h = final(u32(h + torch.arange(nb, device=DEV) * 3266489917))
            h = final(u32(h[own_block] + torch.arange(n, device=DEV) % BLOCK * 2654435761))
            um, uv = (h % 65536 + 0.5) / 65536.0, (torch.div(h, 65536, rounding_mode="floor") + 0.5) / 65536.0
            um, uv = um.double(), uv.double()
            top = lambda x: torch.zeros(nb, dtype=torch.float64, device=DEV).scatter_reduce_(  # noqa: E731
                0, own_block, x, "amax").float().double()[own_block]
            sm, sv = top(m.abs()), top(v)
            y = (m.abs() / sm * 16129).clamp(max=16129)
            k = y.sqrt().floor()
            k = torch.where((y - k.square()) / (2 * k + 1) > um, k + 1, k)
            m = sm * torch.sign(m) * (k / 127).square()
            y = (v / sv * 255.0 ** 4).clamp(max=255.0 ** 4)
            k = y.sqrt().sqrt().floor()
            lo, hi = k.square().square(), (k + 1).square().square()
            k = torch.where((y - lo) / (hi - lo) > uv, k + 1, k)
            v = sv * (torch.where(v > 0, k.clamp(min=1), k) / 255).square().square()
        for name, val in (("p", w), ("master", w), ("m", m), ("v", v)):
            if name in out:
                out[name][cut] = val.to(out[name].dtype)
    return out


def exact(c, seed):
    return {"route": _exact_route, "sgmmb": _exact_sgmmb, "adamw": _exact_adamw}[c["op"]](c, seed)
