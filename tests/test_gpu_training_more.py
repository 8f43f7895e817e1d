"""Training steps over a frozen base in 8 bits, with the balance loss and the orthogonalised momentum: the
operators in a run, as AdapterTraining uses them, against the formulas in binary64."""
import numpy as np
import pytest
import torch

import balance_ref
import dynamic_lora_moe_amd as dlm
import int8_ref
import muon_ref
from dynamic_lora_moe_amd.training import AdapterTraining

pytestmark = pytest.mark.gpu
U = 2.0 ** -24

T, E, R, SCALE, D = 96, 8, 8, 2.0, 64
SHAPES = [(64, D), (136, D), (D, 136)]
READS = [0, 0, 1]  # the first two projections read one input


def _setup(dtype, seed=3):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda std, *s: (torch.randn(s, generator=gen) * std).to(dtype)  # noqa: E731
    x = [rnd(1.0, T, D), rnd(1.0, T, 136)]
    As = [rnd(i ** -0.5, E, R, i) for o, i in SHAPES]
    Bs = [rnd(0.2, E, o, R) for o, i in SHAPES]
    dys = [rnd(1.0, T, o) for o, i in SHAPES]
    W = [torch.randn((o, i), generator=gen) * i ** -0.5 for o, i in SHAPES]
    return x, As, Bs, dys, W, rnd(1.0, T, D), rnd(0.3, D, E)


def _formula(x, As, Bs, x_r, W_r, idx, score, renorm):
    """(the adapters' share of every y, the weights) from leaves, for a given choice."""
    l = x_r @ W_r
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    w = s.gather(1, idx.long())
    g = w / w.sum(1, keepdim=True) if renorm else w
    ys = []
    for r, A, B in zip(READS, As, Bs):
        u = (A[idx.long()] * x[r][:, None, None, :]).sum(3)
        ys.append(SCALE * (g[:, :, None] * (B[idx.long()] * u[:, :, None, :]).sum(3)).sum(1))
    return ys, l


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm,offsets", [("softmax", True, None), ("sigmoid", False, [0, 10, 10, 75, 96])])
def test_steps_over_a_base(dtype, score, renorm, offsets):
    x, As, Bs, dys, W, x_r, W_r = _setup(dtype)
    up = lambda ts: [t.cuda() for t in ts]  # noqa: E731
    dx = [torch.empty_like(t).cuda() for t in x]
    dev_x, dA, dB, ys = up(x), up(As), up(Bs), [torch.empty_like(t).cuda() for t in dys]
    dx_r = torch.zeros_like(x_r).cuda()
    base = [dlm.quantize_rows(w.cuda()) for w in W]
    alpha, zeta = 0.5, 0.01 if score == "softmax" else 0.0
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    tr = AdapterTraining([(dev_x[r], a, b, y) for r, a, b, y in zip(READS, dA, dB, ys)], (x_r.cuda(), W_r.cuda()), up(dys),
                         [dx[r] for r in READS], E, R, SCALE, dx_r=dx_r, score=score, renorm=renorm, base=base, optimizer="muon",
                         weight_decay=0.1, alpha=alpha, zeta=zeta, offsets=off)
    hw = [(q.cpu(), s.cpu()) for q, s in base]
    half = torch.finfo(dtype).eps / 2
    # the bounds of the training operators' own run: fp32 sums, two-term splits, the values' rounding;
    # the base's share is rounded before the adapters join it, once for every projection that shares a dx
    near = lambda a, b, tol: (a.cpu().double() - b).norm() <= tol * b.norm() + 1e-12  # noqa: E731
    for _ in range(2):
        dx_r.zero_()
        for t in ys + dx:
            t.fill_(float("nan"))  # both are written
        before = [m.clone() for m in tr.opt.states]
        weights = [w.clone() for w in (tr.masters or tr.opt.params)]
        idx, _ = tr.forward()
        tr.backward()
        torch.cuda.synchronize()
        leaf = lambda t: t.detach().cpu().double().requires_grad_(True)  # noqa: E731
        lx, lA, lB = [leaf(t) for t in x], [leaf(t) for t in dA], [leaf(t) for t in dB]
        lr_, lW = leaf(x_r), leaf(tr.W_r)
        add, l = _formula(lx, lA, lB, lr_, lW, idx.cpu(), score, renorm)
        sum((y * dy.double()).sum() for y, dy in zip(add, dys)).backward(retain_graph=True)
        loss, counts, rows, _ = balance_ref.balance(l.detach(), idx.cpu(), score, alpha, zeta, offsets)
        dl, _ = balance_ref.backward(l.detach(), counts, rows, 2, score, alpha, zeta, offsets)
        l.backward(dl)  # the balance loss's share of x_r's and W_r's gradients
        assert torch.equal(tr.slots.cpu().long(), counts) and near(tr.loss, loss, 2.0 ** -18)
        for k, r in enumerate(READS):
            assert near(ys[k], int8_ref.forward(x[r], *hw[k]) + add[k].detach(), 2 * half + 2.0 ** -12), k
            assert near(tr.dA[k], lA[k].grad, 2.0 ** -12) and near(tr.dB[k], lB[k].grad, 2.0 ** -12)
        for r in (0, 1):
            mine = [k for k in range(3) if READS[k] == r]
            share = int8_ref.backward([dys[k] for k in mine], [hw[k][0] for k in mine], [hw[k][1] for k in mine])
            assert near(dx[r], share + lx[r].grad, (1 + len(mine)) * half + 2.0 ** -12), r
        assert near(tr.dW_r, lW.grad, 2.0 ** -12) and near(dx_r, lr_.grad, half + 2.0 ** -12)
        # the step, from the gradients the kernels made
        grads = [g.clone() for g in tr.opt.grads]
        tr.step(1e-2)
        assert tr.status() == dlm.DLM_OK
        for k, (w0, m0, g) in enumerate(zip(weights, before, grads)):
            shape = (-1,) + tuple(w0.shape[-2:])
            m, u = muon_ref.momentum(g.cpu().numpy().reshape(shape), m0.cpu().numpy().reshape(shape), 0.95, True)
            new = (tr.masters or tr.opt.params)[k].detach().cpu().double().numpy().reshape(shape)
            for e in range(m.shape[0]):
                xo = muon_ref.by_values(u[e].astype(np.float64), np.float64(np.float32(1e-7)), [muon_ref.COEFS] * 5)
                s = 0.2 * max(shape[1:]) ** 0.5 * 1e-2
                old = w0.cpu().double().numpy().reshape(shape)[e]
                # roundings of the weight and of the update, and the sums' (see the step's own tests)
                tol = 4 * U * np.abs(old) + s * (8 * U * np.abs(xo) + 1e-8 * max(np.abs(xo).max(), 1e-30))
                assert (np.abs(new[e] - (old * (1 - 1e-3) - s * xo)) <= tol + 2 * U * 1e-3 * np.abs(old)).all(), (k, e)
    tr.close()


def _trainer(seed, **kw):
    x, As, Bs, dys, W, x_r, W_r = _setup(torch.bfloat16, seed)
    dx = [torch.empty_like(t).cuda() for t in x]
    dev_x, ys = [t.cuda() for t in x], [torch.empty_like(t).cuda() for t in dys]
    proj = [(dev_x[r], a.cuda(), b.cuda(), y) for r, a, b, y in zip(READS, As, Bs, ys)]
    tr = AdapterTraining(proj, (x_r.cuda(), W_r.cuda()), [t.cuda() for t in dys], [dx[r] for r in READS], E, R, SCALE,
                         base=[dlm.quantize_rows(w.cuda()) for w in W], **kw)
    return tr, ys + dx


@pytest.mark.parametrize("optimizer", ["adamw", "muon"])
@pytest.mark.parametrize("how", ["graph", "stream"])
def test_the_composed_step_replayed_or_on_another_stream(how, optimizer):
    """Replays with eager work between them, or calls on a stream of their own, equal eager calls bit for bit."""
    res = []
    off = torch.tensor([0, 40, 90], dtype=torch.int32, device="cuda")
    for other in (False, True):
        tr, outs = _trainer(7, optimizer=optimizer, alpha=0.1, zeta=1e-3, offsets=off)

        def step():
            tr.forward()
            tr.backward()
            tr.step(1e-2)

        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        if other and how == "stream":
            with torch.cuda.stream(stream):
                for _ in range(4):
                    step()
        elif other:
            with torch.cuda.stream(stream):
                step()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for _ in range(3):
                graph.replay()
                torch.cuda.synchronize()
                torch.zeros(5000, device="cuda").add_(1).sum()
                torch.cuda.synchronize()
        else:
            for _ in range(4):
                step()
        torch.cuda.synchronize()
        assert tr.status() == dlm.DLM_OK
        res.append([*tr.opt.params, *tr.masters, *tr.opt.grads, *outs, tr.loss, tr.slots, tr.rows, tr.probs])
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("scale", ["shape", "rms", 0.5])
def test_update_factors(scale):
    """"shape" is sqrt(max(1, outputs / inputs)) of the map that a matrix is: A [r][d_in] and B [d_out][r] have their
    outputs first, the router's weight [d][E] its inputs."""
    tr, _ = _trainer(5, optimizer="muon", muon_scale=scale, weight_decay=0.0)
    tr.forward()
    tr.backward()
    weights, grads = [w.clone() for w in tr.masters], [g.clone() for g in tr.opt.grads]
    tr.step(1e-2)
    torch.cuda.synchronize()
    assert tr.status() == dlm.DLM_OK
    maps = [m for o, i in SHAPES for m in ((R, i), (o, R))] + [(E, D)]  # (outputs, inputs)
    for k, (w0, g, (o, i)) in enumerate(zip(weights, grads, maps)):
        shape = (-1,) + tuple(w0.shape[-2:])
        g = g.cpu().numpy().reshape(shape)
        _, u = muon_ref.momentum(g, np.zeros_like(g), 0.95, True)
        new, old = (t.cpu().double().numpy().reshape(shape) for t in (tr.masters[k], w0))
        s = 1e-2 * {"shape": max(1.0, o / i) ** 0.5, "rms": 0.2 * max(o, i) ** 0.5}.get(scale, scale)
        for e in range(g.shape[0]):
            x = muon_ref.by_values(u[e].astype(np.float64), np.float64(np.float32(1e-7)), [muon_ref.COEFS] * 5)
            # as for the steps over a base
            tol = 4 * U * np.abs(old[e]) + s * (8 * U * np.abs(x) + 1e-8 * max(np.abs(x).max(), 1e-30))
            assert (np.abs(new[e] - (old[e] - s * x)) <= tol).all(), (k, e)
    tr.close()


@pytest.mark.parametrize("default", [torch.float64, torch.bfloat16])
def test_torchs_default_dtype_does_not_matter(default):
    """What is made here for the caller (momentum, scales, gradients, losses) names its type."""
    res = []
    for kind in (torch.float32, default):
        x, As, Bs, dys, W, x_r, W_r = [[u.cuda() for u in t] if isinstance(t, list) else t.cuda() for t in _setup(torch.bfloat16)]
        dx, ys = [torch.empty_like(t) for t in x], [torch.empty_like(t) for t in dys]
        p8, g8 = torch.ones(1000, device="cuda"), torch.linspace(-1, 1, 1000, device="cuda")
        torch.set_default_dtype(kind)
        try:
            tr = AdapterTraining([(x[r], a, b, y) for r, a, b, y in zip(READS, As, Bs, ys)], (x_r, W_r), dys, [dx[r] for r in READS],
                                 E, R, SCALE, base=[dlm.quantize_rows(w) for w in W], optimizer="muon", alpha=0.1, zeta=1e-3)
            opt = dlm.AdamW([p8], [g8], state_bits=8)
            tr.forward()
            tr.backward()
            tr.step(1e-2)
            opt.step(1e-2)
            m, v = opt.read_state(0)
        finally:
            torch.set_default_dtype(torch.float32)
        assert tr.status() == dlm.DLM_OK
        res.append([*tr.opt.params, *tr.opt.states, *ys, *dx, tr.loss, m, v])
    assert all(a.dtype == b.dtype and torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("grads", ["none", "some", "all"])
def test_a_base_with_longer_buffers_and_unwanted_gradients(grads):
    """Buffers that hold more rows than the batch (x_r's), dys from an iterator, and dxs that are not wanted: the
    same rows as from buffers of the batch's size, and nothing behind them."""
    more, res = 13, []
    for extra in (0, more):
        x, As, Bs, dys, W, x_r, W_r = [[u.cuda() for u in t] if isinstance(t, list) else t.cuda() for t in _setup(torch.bfloat16)]
        longer = lambda t: torch.cat([t, torch.full((extra, t.shape[1]), 2.0, dtype=t.dtype, device="cuda")])  # noqa: E731
        x, dys = [longer(t) for t in x], [longer(t) for t in dys]
        ys, dx = [torch.full_like(t, 3.0) for t in dys], [torch.full_like(t, 3.0) for t in x]
        dxs = None if grads == "none" else [dx[r] if grads == "all" or r == 1 else None for r in READS]
        tr = AdapterTraining([(x[r], a, b, y) for r, a, b, y in zip(READS, As, Bs, ys)], (x_r, W_r), iter(dys),
                             dxs if dxs is None else iter(dxs), E, R, SCALE, base=[dlm.quantize_rows(w) for w in W])
        tr.forward()
        tr.backward()
        tr.step(1e-2)
        assert tr.status() == dlm.DLM_OK
        for t in ys + dx:
            assert (t[T:] == 3).all()
        for r in (0, 1):
            assert bool((dx[r] == 3).all()) == (grads == "none" or (grads == "some" and r == 0))
        res.append([*tr.opt.params, *tr.opt.grads, *(t[:T].clone() for t in ys + dx)])
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_refusals():
    x, As, Bs, dys, W, x_r, W_r = [[u.cuda() for u in t] if isinstance(t, list) else t.cuda() for t in _setup(torch.bfloat16)]
    proj = [(x[r], a, b, torch.empty_like(dy)) for r, a, b, dy in zip(READS, As, Bs, dys)]
    make = lambda **kw: AdapterTraining(proj, (x_r, W_r), dys, [None] * 3, E, R, SCALE, **kw)  # noqa: E731
    for kw in (dict(optimizer="sgd"), dict(optimizer="muon", state_bits=8), dict(base=[dlm.quantize_rows(W[0])])):
        with pytest.raises(ValueError):
            make(**kw)
