"""The cases by which three more operators of training and serving routed adapters are measured.

  balance  the router's balance loss over packed sequences, with counts per expert, and its gradient
  muon     one step of momentum, orthogonalised by Newton-Schulz products, over many matrices
  int8     the frozen base's products in 8-bit integers, scales per token and output channel, and
           their input gradient

A case is a dict of plain values; prepare() makes its inputs on the GPU from a seed, run() does one
pass: the plain form (elementary torch operations) or, with own set, the framework's calls.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}

# One decoder layer of the 7B-shaped workload: (d_out, d_in) of its seven adapted projections, and
# which of them read one input: q, k and v; o; gate and up; down.
LAYER_7B = [(4096, 4096)] * 4 + [(11008, 4096)] * 2 + [(4096, 11008)]
INPUTS_7B = [0, 0, 0, 1, 2, 2, 3]


def listed():
    return [
        # a short fine-tuning batch over the top-2 adapters: latency is all there is
        {"name": "balance-short", "op": "balance", "T": 256, "E": 8, "k": 2, "score": "softmax", "seqs": 1, "dtype": "f32",
         "masked": 0.0, "pad": 0, "zeta": 0.0, "add": 0},
        # packed sequences of ragged lengths, some empty, with padding rows and unavailable experts; both terms
        {"name": "balance-ragged", "op": "balance", "T": 4099, "E": 60, "k": 6, "score": "softmax", "seqs": 37, "dtype": "bf16",
         "masked": 0.1, "pad": 131, "zeta": 1e-3, "add": 0},
        # a large training batch over many small experts, balanced per sequence, joining the routing's gradient
        {"name": "balance-train", "op": "balance", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "seqs": 8, "dtype": "f32",
         "masked": 0.0, "pad": 0, "zeta": 0.0, "add": 1},
        # one projection's banks and their router, odd sizes, single precision
        {"name": "muon-odd-f32", "op": "muon", "shapes": "5x7x333,5x1001x7,1x333x60", "p": "f32", "master": 0, "g": "f32",
         "idle": 1},
        # one 7B-shaped layer's adapter banks, 14 tensors: bf16 weights with fp32 masters
        {"name": "muon-layer", "op": "muon", "shapes": "7b", "layers": 1, "E": 8, "r": 16, "p": "bf16", "master": 1, "g": "f32",
         "idle": 1},
        # a 70B-shaped projection's banks, 16 adapters of rank 64, and a router over 256 experts
        {"name": "muon-wide", "op": "muon", "shapes": "16x64x8192,16x8192x64,1x8192x256", "p": "bf16", "master": 1, "g": "bf16",
         "idle": 0},
        # every adapter of the 7B-shaped model: 448 tensors, 3584 matrices, 322 million weights
        {"name": "muon-model", "op": "muon", "shapes": "7b", "layers": 32, "E": 8, "r": 16, "p": "bf16", "master": 1, "g": "f32",
         "idle": 0},
        # a single decoded token through one layer's base
        {"name": "int8-token", "op": "int8", "T": 1, "shape": "7b", "n": 1, "dtype": "bf16", "back": 0},
        # a mixed decode batch of 64 rows through it
        {"name": "int8-mixed", "op": "int8", "T": 64, "shape": "7b", "n": 1, "dtype": "bf16", "back": 0},
        # odd sizes in single precision, three projections of one input, with the input's gradient
        {"name": "int8-odd-f32", "op": "int8", "T": 523, "shape": "1001x777", "n": 3, "dtype": "f32", "back": 1},
        # prefill: 4096 tokens through one layer
        {"name": "int8-prefill", "op": "int8", "T": 4096, "shape": "7b", "n": 1, "dtype": "bf16", "back": 0},
        # training: the same tokens forward and back
        {"name": "int8-train", "op": "int8", "T": 4096, "shape": "7b", "n": 1, "dtype": "bf16", "back": 1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "muon", "int8"])
    if op == "balance":
        E, score = _log(rng, 2, 256), rng.choice(["softmax", "sigmoid"])
        return {"op": "balance", "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, E)), "score": score,
                "seqs": _log(rng, 1, 64), "dtype": rng.choice(["f32", "bf16"]), "masked": rng.choice([0.0, 0.1]),
                "pad": rng.choice([0, 5]), "zeta": rng.choice([0.0, 1e-3]) if score == "softmax" else 0.0,
                "add": rng.randint(0, 1)}
    if op == "muon":
        shapes = []
        for _ in range(rng.randint(1, 6)):
            small, long = rng.choice([_log(rng, 1, 128), 8, 16, 32, 64]), _log(rng, 8, 8192)
            shapes.append("%dx%dx%d" % ((rng.randint(1, 16),) + rng.choice([(small, long), (long, small)])))
        if rng.randint(0, 2) == 0:
            shapes.append("1x%dx%d" % (_log(rng, 64, 8192), _log(rng, 8, 256)))  # a router's weight
        p = rng.choice(["f32", "bf16"])
        return {"op": "muon", "shapes": ",".join(shapes), "p": p, "master": rng.randint(0, 1) if p == "bf16" else 0,
                "g": rng.choice(["f32", "bf16"]), "idle": rng.randint(0, 1)}
    return {"op": "int8", "T": _log(rng, 1, 4096), "shape": "%dx%d" % (_log(rng, 8, 11008), _log(rng, 8, 11008)),
            "n": rng.randint(1, 3), "dtype": rng.choice(["bf16", "bf16", "f32"]), "back": rng.randint(0, 1)}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def prepare(c, seed):
    return {"balance": _prepare_balance, "muon": _prepare_muon, "int8": _prepare_int8}[c["op"]](c, seed)


def run(s):
    return {"balance": _run_balance, "muon": _run_muon, "int8": _run_int8}[s["c"]["op"]](s)


def work(c):
    if c["op"] == "balance":
        e, n = (4 if c["dtype"] == "f32" else 2), c["T"] * c["E"]
        b = n * e * (3 if c["add"] else 2) + c["T"] * c["k"] * 4 + c["seqs"] * (c["E"] * 8 + 8)
        return {"bytes": b, "flops": 14 * n}
    if c["op"] == "muon":
        p, g, b, f = (4 if c["p"] == "f32" else 2), (4 if c["g"] == "f32" else 2), 0, 0
        for m, rows, cols in _matrices(c):
            n, s = m * rows * cols, min(rows, cols)
            b += n * (g + 8 + (8 + p if c["master"] else 2 * p))
            # the products with the small side's square matrices: once to make one, once to apply one
            f += 4 * n * s + 17 * 2 * m * s ** 3
        return {"bytes": b, "flops": f}
    e, T, b, f, seen = (4 if c["dtype"] == "f32" else 2), c["T"], 0, 0, set()
    for (o, i), x in zip(*_products(c)):
        b += o * i + 4 * o + e * T * o  # the weight, its scales, y
        f += 2 * T * o * i
        if x not in seen:
            b += e * T * i * (2 if c["back"] else 1)  # x, dx
        seen.add(x)
        if c["back"]:
            b += e * T * o  # dy
            f += 2 * T * o * i
    return {"bytes": b, "flops": f}


def exact(c, seed):
    return {"balance": _exact_balance, "muon": _exact_muon, "int8": _exact_int8}[c["op"]](c, seed)


# ------------------------------------------------------------------ balance

ALPHA = 0.01


def _prepare_balance(c, seed):
    g = _gen(seed)
    T, E, S = c["T"], c["E"], c["seqs"]
    # experts of unequal favour, as a router that needs the loss has them
    logits = torch.randn((T, E), generator=g, device=DEV) * 1.5 + torch.randn(E, generator=g, device=DEV)
    if c["masked"]:
        logits = logits.masked_fill(torch.rand((T, E), generator=g, device=DEV) < c["masked"], -math.inf)
    if c["pad"]:
        logits[max(T - c["pad"], 1):] = -math.inf  # padding rows at the end of the last sequence
    logits = logits.to(DT[c["dtype"]])
    top = logits.float().topk(c["k"], 1)
    s = {"c": c, "logits": logits, "offsets": None, "add": None}
    s["idx"] = torch.where(top.values > -math.inf, top.indices, -1).int()
    if S > 1:  # ragged borders, some of them equal: sequences without rows
        cut = torch.randint(0, T + 1, (S - 1,), generator=g, device=DEV)
        ends = torch.tensor([0, T], device=DEV)
        s["offsets"] = torch.cat([ends[:1], cut, ends[1:]]).sort().values.int()
    if c["add"]:
        s["add"] = (torch.randn((T, E), generator=g, device=DEV) * 1e-4).to(logits.dtype)  # the routing's own gradient
    return s


def _run_balance(s):
    c, logits, idx = s["c"], s["logits"], s["idx"]
    if own:
        import dynamic_lora_moe_amd as dlm

        loss, counts, rows, probs = dlm.balance(logits, idx, score=c["score"], alpha=ALPHA, zeta=c["zeta"], offsets=s["offsets"])
        dl = dlm.balance_backward(logits, counts, rows, c["k"], score=c["score"], alpha=ALPHA, zeta=c["zeta"],
                                  offsets=s["offsets"], dlogits=s["add"], accumulate=bool(c["add"]))
        return {"loss": loss, "counts": counts, "rows": rows, "probs": probs, "dlogits": dl}
    T, E, S, k = c["T"], c["E"], c["seqs"], c["k"]
    l = logits.float()
    live = l > -math.inf
    some = live.any(1, keepdim=True)
    # which sequence a row is of
    at = torch.arange(T, device=DEV)
    seq = torch.zeros(T, dtype=torch.long, device=DEV) if S == 1 else (at[:, None] >= s["offsets"][None, 1:S]).sum(1)
    top = torch.where(some, l.amax(1, keepdim=True), 0.0)
    if c["score"] == "softmax":
        sc = torch.exp(l - top)
        tot = sc.sum(1, keepdim=True)
        slope = 1.0
    else:
        sc = 1 / (1 + torch.exp(-l))
        tot = sc.sum(1, keepdim=True)
        slope = 1 - sc
    p = torch.where(some, sc / torch.where(some, tot, 1.0), 0.0)
    rows = torch.zeros(S, device=DEV).index_add_(0, seq, some[:, 0].float())
    n = rows.clamp(min=1.0)[:, None]
    probs = torch.zeros((S, E), device=DEV).index_add_(0, seq, p) / n
    hot = torch.zeros((T, E), device=DEV).scatter_add_(1, idx.long().clamp(min=0), (idx >= 0).float())
    counts = torch.zeros((S, E), device=DEV).index_add_(0, seq, hot * live)
    f = counts * E / (k * n)
    lse = torch.where(some, top + torch.log(torch.where(some, tot, 1.0)), 0.0)[:, 0]
    z = torch.zeros(S, device=DEV).index_add_(0, seq, lse * lse) / n[:, 0]
    loss = torch.stack([ALPHA * (f * probs).sum() / S, c["zeta"] * z.sum() / S])
    u = (ALPHA / S * f / n)[seq]
    dl = p * slope * (u - (u * p).sum(1, keepdim=True))
    if c["zeta"]:
        dl = dl + (2 * c["zeta"] / S) * (lse / n[seq, 0])[:, None] * p
    dl = torch.where(live, dl, 0.0)
    if c["add"]:
        s["add"].copy_(s["add"].float() + dl)
        dl = s["add"]
    return {"loss": loss, "counts": counts.int(), "rows": rows.int(), "probs": probs, "dlogits": dl.to(logits.dtype)}


def _exact_balance(c, seed):
    s = _prepare_balance(c, seed)
    T, E, S, k = c["T"], c["E"], c["seqs"], c["k"]
    l = s["logits"].double()
    dead = torch.isneginf(l)
    none = dead.all(1)
    z = l.masked_fill(dead, 0.0).requires_grad_(True)
    zz = z.masked_fill(dead, -math.inf).masked_fill(none[:, None], 0.0)
    if c["score"] == "softmax":
        p = torch.softmax(zz, 1)
    else:
        sg = torch.sigmoid(zz).masked_fill(dead, 0.0)
        p = sg / sg.sum(1, keepdim=True).masked_fill(none[:, None], 1.0)
    p = p.masked_fill(none[:, None], 0.0)
    lse = torch.logsumexp(zz, 1).masked_fill(none, 0.0)
    border = [0, T] if S == 1 else s["offsets"].tolist()
    bal, zl, counts, rows, probs = 0.0, 0.0, [], [], []
    for a, b in zip(border[:-1], border[1:]):
        m = int((~none[a:b]).sum())
        of = torch.bincount(s["idx"][a:b].flatten().long() + 1, minlength=E + 1)[1:]
        mean = p[a:b].sum(0) / max(m, 1)
        bal = bal + ALPHA / S * E / (k * max(m, 1)) * (of.double() * mean).sum()
        zl = zl + c["zeta"] / S / max(m, 1) * lse[a:b].square().sum()
        counts.append(of)
        rows.append(m)
        probs.append(mean.detach())
    (bal + zl).backward()
    dl = z.grad if s["add"] is None else z.grad + s["add"].double()
    return {"loss": torch.stack([bal.detach(), zl.detach()]), "counts": None, "rows": None, "probs": torch.stack(probs), "dlogits": dl}


# ------------------------------------------------------------------ muon

LR, BETA, WD, EPS = 0.02, 0.95, 0.01, 1e-7
STEPS, COEFS = 5, (3.4445, -4.7750, 2.0315)


def _matrices(c):
    """(matrices, rows, columns) of every tensor: A [E][r][d_in] and B [E][d_out][r] of every projection, or as listed."""
    if c["shapes"] == "7b":
        return [v for _ in range(c["layers"]) for o, i in LAYER_7B for v in ((c["E"], c["r"], i), (c["E"], o, c["r"]))]
    return [tuple(int(v) for v in t.split("x")) for t in c["shapes"].split(",")]


def _prepare_muon(c, seed):
    g = _gen(seed)
    shapes = _matrices(c)
    first = [0]
    for m, rows, cols in shapes:
        first.append(first[-1] + -(-m * rows * cols // 64) * 64)
    # every tensor starts at a multiple of 64 elements of one flat buffer; what lies behind its end is zero
    flat = lambda dt: torch.zeros(first[-1], dtype=dt, device=DEV)  # noqa: E731
    cut = lambda f: None if f is None else [f[a:a + m * r * n].view(m, r, n) for a, (m, r, n) in zip(first, shapes)]  # noqa: E731
    s = {"c": c, "lr": LR, "p": flat(DT[c["p"]]), "g": flat(DT[c["g"]]), "m": flat(torch.float32),
         "master": flat(torch.float32) if c["master"] else None}
    s["of"] = {k: cut(s[k]) for k in ("p", "g", "m", "master")}
    for k, (m, rows, cols) in enumerate(shapes):
        n = min(rows, cols)
        # directions of unequal strength, two decades apart
        fall = torch.logspace(0, -2, n, device=DEV)
        fall = fall[:, None] if rows == n else fall[None, :]
        w = torch.randn((m, rows, cols), generator=g, device=DEV) * 0.02
        s["of"]["m"][k].copy_(torch.randn((m, rows, cols), generator=g, device=DEV) * 3e-4 * fall)
        s["of"]["g"][k].copy_(torch.randn((m, rows, cols), generator=g, device=DEV) * 1e-3 * fall)
        s["of"]["p"][k].copy_(w)
        if c["master"]:
            s["of"]["master"][k].copy_(w)
        if c["idle"] and m > 1:  # an expert that no row has chosen
            s["of"]["g"][k][-1] = 0.0
            s["of"]["m"][k][-1] = 0.0
    if own:
        import dynamic_lora_moe_amd as dlm

        s["opt"] = dlm.Muon(s["of"]["p"], s["of"]["g"], masters=s["of"]["master"], states=s["of"]["m"], momentum=BETA,
                            nesterov=True, weight_decay=WD, eps=EPS, steps=STEPS, coefs=COEFS, scale="shape")
    return s


def _out_muon(s):
    return {"p": s["p"], "m": s["m"]} | ({"master": s["master"]} if s["c"]["master"] else {})


def _run_muon(s):
    if own:
        s["opt"].step(s["lr"])
        return _out_muon(s)
    a, b, c = COEFS
    of = s["of"]
    for p, g, m, master in zip(of["p"], of["g"], of["m"], of["master"] or [None] * len(of["p"])):
        rows, cols = p.shape[1:]
        m.mul_(BETA).add_(g.float(), alpha=1 - BETA)
        x = m * BETA + g.float() * (1 - BETA)
        if rows > cols:
            x = x.transpose(1, 2).contiguous()
        x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
        for _ in range(STEPS):
            q = x @ x.transpose(1, 2).contiguous()
            x = a * x + (b * q + c * (q @ q)) @ x
        if rows > cols:
            x = x.transpose(1, 2)
        w = p.float() if master is None else master
        w = w * (1 - LR * WD) - LR * math.sqrt(max(1.0, rows / cols)) * x
        p.copy_(w)
        if master is not None:
            master.copy_(w)
    return _out_muon(s)


def _exact_muon(c, seed):
    global own
    was, own = own, False
    s = _prepare_muon(c, seed)
    own = was
    out = {k: torch.zeros(v.numel(), dtype=torch.float64, device=DEV) for k, v in _out_muon(s).items()}
    for k, (p, g) in enumerate(zip(s["of"]["p"], s["of"]["g"])):
        w = s["of"]["master" if c["master"] else "p"][k].double()
        m = s["of"]["m"][k].double()
        m = m + (1 - BETA) * (g.double() - m)
        u = m + (1 - BETA) * (g.double() - m)
        wide = u.shape[1] <= u.shape[2]
        u = u if wide else u.transpose(1, 2).contiguous()
        # the step's polynomial acts on the singular values: with u u^T = V diag(v^2) V^T it is
        # V diag(f(v) / v) V^T u
        lam, V = torch.linalg.eigh((u @ u.transpose(1, 2).contiguous()).cpu())
        norm = u.flatten(1).norm(dim=1).cpu()[:, None] + EPS
        t = lam.clamp(min=0).sqrt() / norm
        ratio = 1 / norm + 0 * t
        for _ in range(STEPS):
            by = COEFS[0] + COEFS[1] * t ** 2 + COEFS[2] * t ** 4
            t, ratio = t * by, ratio * by
        P = (V * ratio[:, None, :]) @ V.transpose(1, 2).contiguous()
        x = P.to(DEV) @ u
        x = x if wide else x.transpose(1, 2)
        w = w - LR * WD * w - LR * max(1.0, x.shape[1] / x.shape[2]) ** 0.5 * x
        for name, v in (("p", w), ("m", m), ("master", w)):
            if name in out:
                at = p.storage_offset()
                out[name][at:at + v.numel()] = v.reshape(-1)
    return out


# ------------------------------------------------------------------ int8

def _products(c):
    """The (d_out, d_in) of every product, and the input that it reads."""
    if c["shape"] == "7b":
        n = c["n"]
        return LAYER_7B * n, [4 * j + x for j in range(n) for x in INPUTS_7B]
    o, i = (int(v) for v in c["shape"].split("x"))
    return [(o, i)] * c["n"], [0] * c["n"]


def _prepare_int8(c, seed):
    g, dt, T = _gen(seed), DT[c["dtype"]], c["T"]
    shapes, reads = _products(c)
    s = {"c": c, "reads": reads, "x": {}, "w": [], "sw": [], "y": [], "dy": [], "dx": {}}
    for (o, i), x in zip(shapes, reads):
        if x not in s["x"]:
            # channels of unequal size, as activations have them
            s["x"][x] = (torch.randn((T, i), generator=g, device=DEV) * torch.exp(torch.randn(i, generator=g, device=DEV))).to(dt)
            s["dx"][x] = torch.empty((T, i), dtype=dt, device=DEV)
        s["w"].append((torch.randn((o, i), generator=g, device=DEV) * 36).round().clamp(-127, 127).to(torch.int8))
        s["sw"].append((torch.rand(o, generator=g, device=DEV) + 0.5) * (0.02 / 36))
        s["y"].append(torch.empty((T, o), dtype=dt, device=DEV))
        s["dy"].append((torch.randn((T, o), generator=g, device=DEV) * 1e-3).to(dt) if c["back"] else None)
    if own:
        import dynamic_lora_moe_amd as dlm

        s["grp"] = dlm.Int8Group([(s["x"][x], w, sw, y) for x, w, sw, y in zip(reads, s["w"], s["sw"], s["y"])])
        s["ws"] = s["grp"].workspace(T)
        if c["back"]:
            s["grp"].bind_grads(s["dy"], [s["dx"][x] for x in reads])
            s["wb"] = s["grp"].backward_workspace(T)
    return s


def _codes(v):
    """Whole numbers of -127..127 for each row and what one of them stands for: 127 for the row's largest, halves
    towards zero (64 bits: a value next to a half)."""
    v = v.double()
    top = v.abs().amax(1, keepdim=True)
    at = v.abs() * 127 / torch.where(top > 0, top, 1.0)
    return (torch.ceil(at - 0.5) * torch.sign(v)).float(), (top / 127).float()


def _run_int8(s):
    c = s["c"]
    if own:
        s["grp"].run(workspace=s["ws"])
        if not c["back"]:
            return {"y": s["y"]}
        s["grp"].backward(workspace=s["wb"])
        return {"y": s["y"], "dx": list(s["dx"].values())}
    codes = {x: _codes(v) for x, v in s["x"].items()}
    for x, w, sw, y in zip(s["reads"], s["w"], s["sw"], s["y"]):
        q, sx = codes[x]
        y.copy_((q @ w.float().t()) * sx * sw)
    if not c["back"]:
        return {"y": s["y"]}
    for x, dx in s["dx"].items():
        # every channel that reads x, side by side, each with its scale: one row of codes for a token
        mine = [k for k, v in enumerate(s["reads"]) if v == x]
        q, sd = _codes(torch.cat([s["dy"][k].double() * s["sw"][k].double() for k in mine], 1))
        dx.copy_((q @ torch.cat([s["w"][k].float() for k in mine])) * sd)
    return {"y": s["y"], "dx": list(s["dx"].values())}


def _exact_int8(c, seed):
    global own
    was, own = own, False
    s = _prepare_int8(c, seed)
    own = was

    def whole(v):
        r = v.abs().max(dim=1, keepdim=True).values
        t = torch.nan_to_num(v.abs() / r * 127)
        up = torch.floor(t)
        return torch.where(t - up > 0.5, up + 1, up).copysign(v), r / 127

    out = {"y": []}
    for x, w, sw in zip(s["reads"], s["w"], s["sw"]):
        q, r = whole(s["x"][x].double())
        out["y"].append(r * (q @ (w.double() * sw.double()[:, None]).t()))
    if c["back"]:
        out["dx"] = []
        for x in s["dx"]:
            mine = [k for k in range(len(s["w"])) if s["reads"][k] == x]
            q, r = whole(torch.cat([s["dy"][k].double() * s["sw"][k].double() for k in mine], 1))
            done = torch.zeros_like(s["dx"][x], dtype=torch.float64)
            at = 0
            for k in mine:
                done += q[:, at:at + s["w"][k].shape[0]] @ s["w"][k].double()
                at += s["w"][k].shape[0]
            out["dx"].append(done * r)
    return out
