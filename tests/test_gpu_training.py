"""The training operators in a run: routing, the adapters' product, its gradients,
the router's gradient and the AdamW step, as one training step uses them.  The
gradients are held to autograd of the formulas in binary64, with the routing's
choice fixed; every bound counts the roundings on the way."""
import numpy as np
import pytest
import torch

import adamw_ref
import dynamic_lora_moe_amd as dlm
from dynamic_lora_moe_amd.training import AdapterTraining

pytestmark = pytest.mark.gpu


def _formula(xs, As, Bs, x_r, W_r, idx, scale, score, renorm):
    """(every y, dtype binary64) from leaves, for a given choice."""
    l = x_r @ W_r
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    w = s.gather(1, idx.long())
    g = w / w.sum(1, keepdim=True) if renorm else w
    ys = []
    for x, A, B in zip(xs, As, Bs):
        u = torch.einsum("ti,tkri->tkr", x, A[idx.long()])
        ys.append(scale * torch.einsum("tk,tkr,tkor->to", g, u, B[idx.long()]))
    return ys, g


@pytest.mark.parametrize("dtype,bits", [(torch.float32, 32), (torch.float32, 8), (torch.bfloat16, 32), (torch.bfloat16, 8)])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("sigmoid", False)])
def test_steps_of_the_adapters(dtype, bits, score, renorm):
    T, E, r, scale, d = 96, 8, 8, 2.0, 64
    shapes = [(64, d), (136, d), (d, 136)]
    gen = torch.Generator().manual_seed(3)
    rnd = lambda std, *s: (torch.randn(s, generator=gen) * std).to(dtype)  # noqa: E731
    xs = [rnd(1.0, T, i) for o, i in shapes]
    As = [rnd(i ** -0.5, E, r, i) for o, i in shapes]
    Bs = [rnd(0.2, E, o, r) for o, i in shapes]
    dys = [rnd(1.0, T, o) for o, i in shapes]
    x_r, W_r = rnd(1.0, T, d), rnd(0.3, d, E)
    up = lambda ts: [t.cuda() for t in ts]  # noqa: E731
    dxs, ys = [torch.zeros_like(x).cuda() for x in xs], [torch.zeros_like(t).cuda() for t in dys]
    dx_r = torch.zeros_like(x_r).cuda()
    dA, dB = up(As), up(Bs)
    proj = list(zip(up(xs), dA, dB, ys))
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    tr = AdapterTraining(proj, (x_r.cuda(), W_r.cuda()), up(dys), dxs, E, r, scale, dx_r=dx_r, score=score, renorm=renorm,
                         counts=counts, state_bits=bits, weight_decay=0.0, seed=1)
    half = torch.finfo(dtype).eps / 2
    for step in range(3):
        for t in ys + dxs + [dx_r]:
            t.zero_()
        before = [t.clone() for t in tr.opt.params]
        moments = [tuple(x.clone() for x in tr.opt.read_state(k)) for k in range(len(before))]
        masters = None if tr.masters is None else [m.clone() for m in tr.masters]
        idx, g = tr.forward()
        tr.backward()
        torch.cuda.synchronize()
        # autograd of the formulas on the weights as they are now
        leaf = lambda t: t.detach().cpu().double().requires_grad_(True)  # noqa: E731
        lx, lA, lB = [leaf(x) for x in xs], [leaf(t) for t in dA], [leaf(t) for t in dB]
        lr_, lW = leaf(x_r), leaf(tr.W_r)
        want, wg = _formula(lx, lA, lB, lr_, lW, idx.cpu(), scale, score, renorm)
        sum((y * dy.double()).sum() for y, dy in zip(want, dys)).backward()
        # fp32 sums of up to 136 * 8 products, and 96 rows for the banks: 2^-24 times their number, of the
        # sum of magnitudes, bounded by its root mean square times the terms; far below 2^-12 of the norm,
        # which bf16's two-term splits (2^-16), fp32 logits (2^-24 d) and the values' own rounding stay under
        near = lambda a, b, tol: (a.cpu().double() - b).norm() <= tol * b.norm() + 1e-12  # noqa: E731
        assert near(g, wg.detach(), 2.0 ** -20)
        for k in range(3):
            assert near(ys[k], want[k].detach(), half + 2.0 ** -12), (step, k, "y")
            assert near(dxs[k], lx[k].grad, half + 2.0 ** -12), (step, k, "dx")
            assert near(tr.dA[k], lA[k].grad, 2.0 ** -12), (step, k, "dA")
            assert near(tr.dB[k], lB[k].grad, 2.0 ** -12), (step, k, "dB")
        assert near(tr.dW_r, lW.grad, 2.0 ** -12) and near(dx_r, lr_.grad, half + 2.0 ** -12)
        # the step, from the gradients the kernels made
        tr.step(1e-2)
        assert tr.status() == dlm.DLM_OK
        for k, (p0, (m0, v0)) in enumerate(zip(before, moments)):
            f = lambda t: t.detach().cpu().double().numpy().ravel()  # noqa: E731
            m, v = adamw_ref.moments(f(tr.opt.grads[k]), f(m0), f(v0), 0.9, 0.999)
            w = f(p0 if masters is None else masters[k])
            new, s = adamw_ref.update(w, m, v, step + 1, 1e-2, 0.9, 0.999, 1e-8, 0.0)
            got = f(tr.opt.params[k] if masters is None else tr.masters[k])
            # read back as fp32, the 8-bit moments are 2^-24 off what the step had: 2^-22 of the step and 16 of its own roundings
            assert (np.abs(got - new) <= 2.0 ** -22 * np.abs(w) + 1e-2 * (2.0 ** -18) * np.maximum(np.abs(s), 1.0)).all()
    assert int(counts.sum()) == 3 * T * 2
    tr.close()


def test_padding_rows_reach_nothing():
    """Tokens whose logits are all -inf (padding): no adapter, no gradient, whatever their rows hold."""
    T, E, r, d = 40, 4, 8, 64
    gen = torch.Generator().manual_seed(0)
    x, dy = torch.randn((T, d), generator=gen).bfloat16().cuda(), torch.randn((T, d), generator=gen).bfloat16().cuda()
    A = (torch.randn((E, r, d), generator=gen) * 0.1).bfloat16().cuda()
    B = (torch.randn((E, d, r), generator=gen) * 0.1).bfloat16().cuda()
    logits = torch.randn((T, E), generator=gen).cuda()
    out = []
    for rows in (30, 40):
        xr, dyr = x.clone(), dy.clone()
        lr_ = logits.clone()
        if rows == 40:
            lr_[30:], xr[30:], dyr[30:] = -float("inf"), float("nan"), float("inf")
        xr, dyr, lr_ = xr[:rows].contiguous(), dyr[:rows].contiguous(), lr_[:rows].contiguous()
        y, dx = torch.zeros_like(dyr), torch.zeros_like(xr)
        dA, dB = torch.empty(A.shape, device="cuda"), torch.empty(B.shape, device="cuda")
        dg = torch.empty((rows, 2), device="cuda")
        grp = dlm.SgmmGroup([(xr, A, B, y)], E, r, 1.0)
        grp.bind_grads([dyr], [dx], [dA], [dB])
        idx, g = dlm.route(lr_, 2)
        grp.run(idx, g)
        grp.backward(idx, g, dg)
        dl = dlm.route_backward(lr_, idx, dg)
        torch.cuda.synchronize()
        assert (idx[30:] == -1).all() and (y[30:] == 0).all() and (dx[30:] == 0).all() and (dl[30:] == 0).all()
        out.append([t[:30] if t.shape[0] == rows else t for t in (idx, g, y, dx, dg, dl)] + [dA, dB])
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_a_whole_step_replayed_from_a_graph():
    """Routing to AdamW captured once: replays, with eager work between them, equal eager steps bit for bit."""
    T, E, r, d = 70, 8, 16, 128
    res = []
    for captured in (False, True):
        gen = torch.Generator().manual_seed(5)
        rnd = lambda std, *s: (torch.randn(s, generator=gen) * std).bfloat16().cuda()  # noqa: E731
        x, A, B, dy = rnd(1.0, T, d), rnd(0.1, E, r, d), rnd(0.1, E, d, r), rnd(1.0, T, d)
        y, dx = torch.zeros_like(dy), torch.zeros_like(x)
        logits = torch.randn((T, E), generator=gen).cuda()
        dA, dB = torch.zeros(A.shape, device="cuda"), torch.zeros(B.shape, device="cuda")
        idx, g = dlm.route(logits, 2)
        dg, dl = torch.empty_like(g), torch.empty_like(logits)
        grp = dlm.SgmmGroup([(x, A, B, y)], E, r, 1.0)
        grp.bind_grads([dy], [dx], [dA], [dB])
        ws, wb = grp.workspace(T), grp.backward_workspace(T)
        opt = dlm.AdamW([A, B], [dA, dB], masters=[A.float(), B.float()], state_bits=8, seed=2)

        def step():
            dlm.route(logits, 2, idx=idx, g=g)
            grp.run(idx, g, workspace=ws)
            grp.backward(idx, g, dg, workspace=wb)
            dlm.route_backward(logits, idx, dg, dlogits=dl)
            opt.step(1e-2)
            grp.repack()

        step()
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for _ in range(3):
                graph.replay()
                torch.cuda.synchronize()
                torch.zeros(1000, device="cuda").add_(1)  # eager work between
                torch.cuda.synchronize()
        else:
            for _ in range(3):
                step()
        torch.cuda.synchronize()
        assert opt.status() == (4, dlm.DLM_OK)
        res.append([A, B, y, dx, dA, dB, dg, dl])
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.fixture
def dirty_workspaces(monkeypatch):
    """Byte tensors that torch.empty makes hold garbage."""
    real = torch.empty

    def empty(*a, **k):
        t = real(*a, **k)
        return t.fill_(0x5A) if t.dtype == torch.uint8 else t

    monkeypatch.setattr(torch, "empty", empty)


def test_status_before_anything_ran(dirty_workspaces):
    """The status is that of the calls so far, whatever the workspaces' memory held."""
    T, E, r, d = 8, 4, 8, 64
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    tr = AdapterTraining([(z(T, d), z(E, r, d), z(E, d, r), z(T, d))], (z(T, d), z(d, E)), [z(T, d)], [z(T, d)], E, r, 1.0)
    assert tr.status() == dlm.DLM_OK
    tr.forward()
    assert tr.status() == dlm.DLM_OK
    tr.backward()
    tr.step(1e-3)
    assert tr.status() == dlm.DLM_OK


def test_status_of_calls_without_rows(dirty_workspaces):
    E, r, d = 4, 8, 64
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    grp = dlm.SgmmGroup([(z(8, d), z(E, r, d), z(E, d, r), z(8, d))], E, r, 1.0)
    grp.bind_grads([z(8, d)], [z(8, d)], [torch.empty((E, r, d), device="cuda")], [torch.empty((E, d, r), device="cuda")])
    idx, g = torch.zeros((8, 2), dtype=torch.int32, device="cuda"), torch.zeros((8, 2), device="cuda")
    for call in (grp.run, grp.backward):
        assert dlm.sgmm_status(call(idx, g, T=0)) == dlm.DLM_OK


@pytest.mark.parametrize("how", ["graph", "stream"])
def test_the_composed_step_replayed_or_on_another_stream(how):
    """AdapterTraining's own step, router products included: replays with eager work between them, or calls on a
    stream of their own, equal eager calls bit for bit."""
    T, E, r, d = 200, 8, 16, 128
    shapes = [(64, d), (136, d), (d, 136)]
    res = []
    for other in (False, True):
        gen = torch.Generator().manual_seed(7)
        rnd = lambda std, *s: (torch.randn(s, generator=gen) * std).bfloat16().cuda()  # noqa: E731
        proj = [(rnd(1.0, T, i), rnd(0.1, E, r, i), rnd(0.1, E, o, r), rnd(1.0, T, o)) for o, i in shapes]
        dys, dxs = [rnd(1.0, T, o) for o, _ in shapes], [rnd(1.0, T, i) for _, i in shapes]
        x_r, W_r, dx_r = rnd(1.0, T, d), rnd(0.3, d, E), rnd(1.0, T, d)
        counts = torch.zeros(E, dtype=torch.int32, device="cuda")
        tr = AdapterTraining(proj, (x_r, W_r), dys, dxs, E, r, 1.5, dx_r=dx_r, counts=counts, state_bits=8, seed=3)

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
        assert tr.status() == dlm.DLM_OK and int(counts.sum()) == 4 * 2 * T
        res.append([*tr.opt.params, *tr.masters, *tr.opt.grads, *(p[3] for p in proj), *dxs, dx_r, tr.dg, tr.logits])
    assert all(torch.equal(a, b) for a, b in zip(*res))
