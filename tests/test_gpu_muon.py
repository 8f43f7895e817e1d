"""The orthogonalised momentum step on the GPU against the plain binary64 form.

Tolerances (U = 2^-24).
  m: compared with the same fp32 arithmetic, to the last bit or one beside it (a fused sum that
     binary64 rounds a second time): 2 U |m|.
  X: of the u that those bits give, by singular values in binary64.  The kernel's sums and square
     matrices are binary64: a sum of d products is off by at most d 2^-53 of |u|^2, and each of the K
     steps adds some n 2^-53; the steps raise a weak direction's square and its error by a^2 each, a^2K
     together (2.4e5 for five), and what that does to the last factors is of the order of itself: below
     d 2^-53 2.4e5 < 1e-6 of the strongest entry for d < 4e4 -- and of that the root over the
     entries, as errors do not conspire: 1e-8.  A u off by one rounding in a few elements moves X by
     485 2^-24 of them, below that too.  Then one fp32 rounding, and the update's two: 4 U |X|.
  w: 4 U |w| on top; bf16 parameters are the master's rounding."""
import ctypes as C

import numpy as np
import pytest
import torch

import dynamic_lora_moe_amd as dlm
import muon_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BETA, EPS = 0.95, 1e-7


def _rnd(shape, seed, std=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std


def _f64(t):
    return t.detach().cpu().double().numpy()


def _place(t, shift=0):
    """t on the device, `shift` elements behind an aligned address, with a guard on both sides."""
    buf = torch.full((t.numel() + 64,), 3, dtype=t.dtype, device="cuda")
    v = buf[16 + shift:16 + shift + t.numel()].view(t.shape)
    v.copy_(t)
    return v, buf, shift


def _guards(placed):
    for v, buf, shift in placed:
        assert (buf[:16 + shift] == 3).all() and (buf[16 + shift + v.numel():] == 3).all()


def _compare(p0, w0, m0, g, p, w, m, lr, wd, scale, nesterov=True, coefs=None, gscale=1.0, eps=EPS, beta=BETA):
    coefs = coefs or [ref.COEFS] * 5
    shape = p0.shape
    g, m0 = g.float().cpu().numpy().reshape(-1, *shape[-2:]), m0.cpu().numpy().reshape(-1, *shape[-2:])
    m1, u = ref.momentum(g, m0, beta, nesterov, gscale)
    got_m = m.cpu().numpy().reshape(m1.shape)
    assert (np.abs(got_m.astype(np.float64) - m1) <= 2 * U * np.abs(m1)).all()
    old = _f64(p0 if w0 is None else w0).reshape(m1.shape)
    new = _f64(p if w is None else w).reshape(m1.shape)
    half = torch.finfo(p.dtype).eps / 2 if w is None and p.dtype != torch.float32 else 0.0
    for k in range(m1.shape[0]):
        x = ref.by_values(u[k].astype(np.float64), eps, coefs)
        want = old[k] * (1 - lr * wd) - lr * scale * x
        tol = 4 * U * np.abs(old[k]) + abs(lr * scale) * (4 * U * np.abs(x) + 1e-8 * max(np.abs(x).max(), 1e-30)) + 2.0 ** -140
        err = np.abs(new[k] - want)
        assert (err <= tol + half * (np.abs(want) + tol)).all(), (k, shape, err.max(), np.abs(x).max())
    if w is not None:
        assert torch.equal(p, w.to(p.dtype))


def _run(shapes, p_dtype, g_dtype, master, steps=2, shift=0, make_g=None, lr=0.5, wd=0.0, **kw):
    placed, ps, gs, ms, ws = [], [], [], [], []

    def put(t):
        placed.append(_place(t, shift))
        return placed[-1][0]

    for k, s in enumerate(shapes):
        w = _rnd(s, 10 * k, 0.02)
        ps.append(put(w.to(p_dtype)))
        gs.append(put((make_g(s, k) if make_g else _rnd(s, 10 * k + 1, 1e-3)).to(g_dtype)))
        ms.append(put(_rnd(s, 10 * k + 2, 3e-4)))
        ws.append(put(w) if master else None)
    scales = [1.0 + 0.1 * (k % 3) for k in range(len(shapes))]
    wds = [wd * (k % 2) for k in range(len(shapes))]
    opt = dlm.Muon(ps, gs, masters=ws, states=ms, momentum=BETA, weight_decay=wds, eps=EPS, scale=scales, **kw)
    nest = kw.get("nesterov", True)
    for _ in range(steps):
        snap = [(p.clone(), None if w is None else w.clone(), m.clone()) for p, w, m in zip(ps, ws, ms)]
        opt.step(lr)
        torch.cuda.synchronize()
        for k, (p0, w0, m0) in enumerate(snap):
            _compare(p0, w0, m0, gs[k], ps[k], ws[k], ms[k], lr, wds[k], np.float32(scales[k]).astype(float), nest)
        for g in gs:
            g.mul_(-0.5)
    _guards(placed)
    assert opt.status() == dlm.DLM_OK
    return ps, ms, ws


SHAPES = [(1, 1), (1, 7), (5, 1), (3, 4, 8), (2, 16, 16), (2, 16, 64), (3, 64, 16), (2, 7, 333), (2, 1001, 7), (17, 100), (100, 17),
          (2, 32, 1024), (2, 1028, 32), (33, 70), (64, 64), (2, 64, 520), (2, 1000, 64), (63, 517), (517, 63), (16, 4096), (4100, 16),
          (40, 2000), (2000, 48), (2, 2, 8, 24)]
BIG = [(65, 65), (66, 300), (300, 65), (128, 128), (2, 128, 520), (700, 100), (512, 600), (600, 509), (200, 2000)]
TYPES = [(torch.float32, torch.float32, False), (torch.bfloat16, torch.float32, True), (torch.bfloat16, torch.bfloat16, True),
         (torch.bfloat16, torch.bfloat16, False), (torch.float32, torch.bfloat16, False)]


@pytest.mark.parametrize("p_dtype,g_dtype,master", TYPES)
def test_sizes_and_types(p_dtype, g_dtype, master):
    _run(SHAPES, p_dtype, g_dtype, master, wd=0.1)


@pytest.mark.parametrize("p_dtype,g_dtype,master", TYPES)
def test_small_sides_above_64(p_dtype, g_dtype, master):
    _run(BIG + [(8, 40)], p_dtype, g_dtype, master, wd=0.1)


def test_classes_of_many_pieces():
    """Small sides of every class in more pieces than share launches."""
    _run([(300, 16, 40), (40, 150, 30), (8, 40, 5000), (7, 6000, 60), (300, 9, 7)], torch.bfloat16, torch.float32, True, steps=1)


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_unaligned_tensors(shift):
    """Tensors at any multiple of their element's size: the same results as aligned ones, bit for bit."""
    shapes = [(16, 200), (200, 16), (2, 48, 100), (100, 72), (5, 9)]
    a = _run(shapes, torch.bfloat16, torch.float32, True, shift=shift)
    b = _run(shapes, torch.bfloat16, torch.float32, True)
    assert all(torch.equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))


@pytest.mark.parametrize("shape", [(16, 700), (700, 16), (48, 500), (90, 300), (300, 130)])
@pytest.mark.parametrize("decades", [3, 6, 30])
def test_weak_directions(shape, decades):
    """Directions down to 10^-decades of the strongest (fp32 squares would lose them from 10^-4 on)."""
    def make(s, k):
        n = min(s)
        fall = torch.logspace(0, -decades, n, dtype=torch.float64)
        g = _rnd(s, k).double()
        # rows scaled, then mixed by a rotation, so that no single entry carries a direction
        q, _ = torch.linalg.qr(_rnd((n, n), 7).double())
        g = q @ (fall[:, None] * g) if s[0] == n else (g * fall) @ q.t()
        return g.float()

    for beta in (0.0, BETA):
        p = torch.zeros(shape, device="cuda")
        g, m0 = make(shape, 1).cuda(), make(shape, 2).cuda()
        m = m0.clone()
        opt = dlm.Muon([p], [g], states=[m], momentum=beta, scale=1.0)
        opt.step(1.0)
        _compare(torch.zeros(shape), None, m0, g, p, None, m, 1.0, 0.0, 1.0, beta=beta)


def test_equal_and_missing_directions():
    """Orthogonal rows of one length (every value is 1 / sqrt n), repeated rows, one row, no row at all."""
    g = torch.zeros((4, 24, 96))
    g[0] = torch.eye(24, 96)
    g[1] = _rnd((1, 96), 1).expand(24, 96)
    g[2, 3] = _rnd((96,), 2)
    p = torch.zeros_like(g).cuda()
    m = torch.zeros_like(g).cuda()
    opt = dlm.Muon([p], [g.cuda()], states=[m], scale=1.0)
    opt.step(1.0)
    _compare(torch.zeros(g.shape), None, torch.zeros(g.shape), g, p, None, m, 1.0, 0.0, 1.0)
    assert (p[3] == 0).all() and (m[3] == 0).all() and opt.status() == dlm.DLM_OK


@pytest.mark.parametrize("std", [1e-30, 1e-12, 1e10, 1e18])
def test_sizes_of_gradients(std):
    for shape in ((16, 300), (80, 200)):
        g, p, m = _rnd(shape, 1, std).cuda(), torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
        dlm.Muon([p], [g], states=[m], scale=1.0, eps=1e-38).step(1.0)
        _compare(torch.zeros(shape), None, torch.zeros(shape), g, p, None, m, 1.0, 0.0, 1.0, eps=np.float32(1e-38).astype(float))


@pytest.mark.parametrize("nesterov", [True, False])
def test_without_nesterov_and_other_products(nesterov):
    _run([(16, 300), (3, 50, 40), (300, 70)], torch.float32, torch.float32, False, nesterov=nesterov)
    triples = [(1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (2.0, -1.5, 0.5)]
    for shape in ((12, 80), (80, 130)):
        g, p, m = _rnd(shape, 1).cuda(), torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
        dlm.Muon([p], [g], states=[m], scale=2.0, nesterov=nesterov, steps=3, coefs=triples).step(1.0)
        _compare(torch.zeros(shape), None, torch.zeros(shape), g, p, None, m, 1.0, 0.0, 2.0, nesterov=nesterov, coefs=triples)
        dlm.Muon([p.zero_()], [g], states=[m.zero_()], scale=2.0, nesterov=nesterov, steps=1).step(1.0)
        _compare(torch.zeros(shape), None, torch.zeros(shape), g, p, None, m, 1.0, 0.0, 2.0, nesterov=nesterov, coefs=[ref.COEFS])
        dlm.Muon([p.zero_()], [g], states=[m.zero_()], scale=2.0, nesterov=nesterov, steps=10, coefs=[(1.5, -0.5, 0.0)] * 10).step(1.0)
        _compare(torch.zeros(shape), None, torch.zeros(shape), g, p, None, m, 1.0, 0.0, 2.0, nesterov=nesterov,
                 coefs=[(1.5, -0.5, 0.0)] * 10)


def test_a_matrix_that_is_not_finite_stays():
    """Infinities and NaN in one matrix leave it, momentum too, and its neighbours as they would be without it."""
    shapes = [(3, 16, 100), (3, 100, 40), (3, 70, 90)]
    res = []
    for bad in (False, True):
        ps = [_rnd(s, k, 0.02).cuda() for k, s in enumerate(shapes)]
        gs = [_rnd(s, 9 + k, 1e-3).cuda() for k, s in enumerate(shapes)]
        ms = [_rnd(s, 20 + k, 1e-3).cuda() for k, s in enumerate(shapes)]
        p0, m0 = [p.clone() for p in ps], [m.clone() for m in ms]
        if bad:
            gs[0][1, 3, 4] = float("inf")
            gs[1][1, 99, 39] = float("nan")
            ms[2][1, 0, 0] = -float("inf")
            m0[2] = ms[2].clone()
        opt = dlm.Muon(ps, gs, states=ms)
        opt.step(0.1)
        assert opt.status() == (dlm.DLM_EDEVICE if bad else dlm.DLM_OK) and opt.status() == dlm.DLM_OK
        if bad:
            for p, q, m, n in zip(ps, p0, ms, m0):
                assert torch.equal(p[1], q[1]) and torch.equal(m[1], n[1])
        res.append([t[::2] for t in ps + ms])
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_lr_and_gradient_scales_from_the_device():
    g = _rnd((3, 16, 300), 1, 1e-3).cuda()
    half = torch.tensor([0.5], device="cuda")
    for shape in ((3, 16, 300), (1, 144, 100)):
        a, b = (_rnd(shape, 2, 0.02).cuda() for _ in range(2))
        gg = g.view(shape)
        x, y = dlm.Muon([a], [gg], scale="rms"), dlm.Muon([b], [gg * 0.5], scale="rms")
        for _ in range(2):
            x.step(2e-2, lr_scale=half, grad_scale=half)
            y.step(1e-2)
        assert torch.equal(a, b)


def test_replayed_from_a_graph():
    """Replays with new gradients and rates, with eager work between them, equal eager steps bit for bit."""
    shapes = [(4, 16, 520), (4, 520, 16), (2, 48, 300), (1, 200, 96), (30, 30)]
    sides = []
    for _ in range(2):
        ps = [_rnd(s, k, 0.02).bfloat16().cuda() for k, s in enumerate(shapes)]
        gs = [_rnd(s, 50 + k, 1e-3).cuda() for k, s in enumerate(shapes)]
        ws = [p.float() for p in ps]
        sides.append((ps, gs, ws, dlm.Muon(ps, gs, masters=ws, weight_decay=0.1)))
    lr = torch.tensor([1.0], device="cuda")
    for _, _, _, o in sides:
        o.step(1e-2, lr_scale=lr)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sides[0][3].step(1e-2, lr_scale=lr)
    for k in range(3):
        lr.fill_(1.0 / (k + 1))
        for _, gs, _, _ in sides:
            for g in gs:
                g.mul_(-0.7)
        graph.replay()
        torch.cuda.synchronize()
        sides[1][3].step(1e-2, lr_scale=lr)
        torch.cuda.synchronize()
        for a, b in zip(*[s[0] + s[2] + s[3].states for s in sides]):
            assert torch.equal(a, b)


def test_other_stream_many_tensors_and_fresh_momentum():
    """A hundred tensors on a stream of their own, momentum made behind queued work, against the current stream."""
    shapes = [(1 + k % 3, 1 + (7 * k) % 70, 1 + (37 * k) % 300) for k in range(100)]
    out = []
    for other in (False, True):
        ps = [_rnd(s, k, 0.02).cuda() for k, s in enumerate(shapes)]
        gs = [_rnd(s, 500 + k, 1e-3).cuda() for k, s in enumerate(shapes)]
        torch.cuda.synchronize()
        if other:
            one, two = torch.cuda.Stream(), torch.cuda.Stream()
            with torch.cuda.stream(one):
                torch.cuda._sleep(100_000_000)
                opt = dlm.Muon(ps, gs)
            opt.step(1e-2, stream=two)
        else:
            opt = dlm.Muon(ps, gs)
            opt.step(1e-2)
        torch.cuda.synchronize()
        assert opt.status() == dlm.DLM_OK
        out.append(ps + opt.states)
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_past_2_32_elements():
    """More than 2^32 elements, as many matrices and as one: what matters lies behind 2^32."""
    r, d = 16, 4096
    n = (1 << 32) // (r * d) + 3
    print("muon", n, r, d, flush=True)
    p = torch.zeros((n, r, d), dtype=torch.bfloat16, device="cuda")
    g = torch.zeros((n, r, d), dtype=torch.bfloat16, device="cuda")
    g[-2:] = _rnd((2, r, d), 1, 1e-3).bfloat16().cuda()
    opt = dlm.Muon([p], [g], scale=1.0)
    opt.step(1.0)
    q = torch.zeros((2, r, d), dtype=torch.bfloat16, device="cuda")
    small = dlm.Muon([q], [g[-2:].clone()], scale=1.0)
    small.step(1.0)
    assert torch.equal(p[-2:], q) and torch.equal(opt.states[0][-2:], small.states[0])
    assert not p[:-2].any()
    opt.close()
    del opt, p, g
    torch.cuda.empty_cache()
    for side, wide in ((5, True), (5, False), (65, True)):
        d = (1 << 32) // side + 2048
        shape = (side, d) if wide else (d, side)
        print("muon", shape, flush=True)
        p = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        g = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        tail = _rnd((side, 1024) if wide else (1024, side), 2, 1e-3).bfloat16().cuda()
        cut = (slice(None), slice(d - 1024, d)) if wide else (slice(d - 1024, d),)
        g[cut] = tail
        opt = dlm.Muon([p], [g], scale=1.0)
        opt.step(1.0)
        q = torch.zeros_like(tail)
        dlm.Muon([q], [tail], scale=1.0).step(1.0)
        # the same columns in other pieces: binary64 sums in another order, below half a bf16 step
        diff = (p[cut].double() - q.double()).abs()
        assert (diff <= 2.0 ** -7 * q.double().abs()).all() and (diff > 0).double().mean() < 1e-4
        assert not p[(slice(None), slice(0, 4096)) if wide else slice(0, 4096)].any()
        opt.close()
        del opt, p, g
        torch.cuda.empty_cache()


def test_ten_of_the_default_steps():
    """Twice the usual number of products that raise weak directions.  Directions of one size: the usual bounds.
    (Their error, some 2^-53 / 10^-4 of themselves, grows by 1.7 a step at most once they are near 1.)  Down to
    10^-6 of the strongest: a sum's error, d 2^-53 of |u|^2, and n 2^-53 for each of the square products, are
    raised by a^2 a step, which the singular values of the difference are held to."""
    coefs = [ref.COEFS] * 10
    for shape in ((16, 300), (48, 300), (300, 40), (80, 130)):
        g, p, m = _rnd(shape, 1).cuda(), torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
        dlm.Muon([p], [g], states=[m], scale=1.0, steps=10).step(1.0)
        _compare(torch.zeros(shape), None, torch.zeros(shape), g, p, None, m, 1.0, 0.0, 1.0, coefs=coefs)
        n, d = min(shape), max(shape)
        q, _ = torch.linalg.qr(_rnd((n, n), 7).double())
        fall = torch.logspace(0, -6, n, dtype=torch.float64)
        h = (q @ (fall[:, None] * _rnd((n, d), 2).double())).float()
        h = (h if shape[0] == n else h.t()).contiguous().cuda()
        dlm.Muon([p.zero_()], [h], states=[m.zero_()], scale=1.0, steps=10).step(1.0)
        _, u = ref.momentum(h.cpu().numpy(), np.zeros(shape, np.float32), BETA, True)
        x = ref.by_values(u.astype(np.float64), np.float64(np.float32(EPS)), coefs)
        err = np.linalg.norm(-_f64(p) - x, 2)
        print(shape, err)
        assert err <= ref.growth(coefs) ** 2 * (d + 10 * n) * 2.0 ** -53 + 4 * U * np.linalg.norm(x)


def test_scratch_that_does_not_fit_is_refused_and_leaves_nothing_behind():
    """More scratch memory than the device has (450 GB): the status of a failed allocation, and the next calls,
    of the library and of others, do not find its error."""
    at = 1 << 44
    big = (dlm.dlm_muon_param * 1)(dlm.dlm_muon_param(at, 2 * at, None, 3 * at, 1, 512, 1 << 26, 0.0, 1.0))
    h = C.c_void_p()
    p, g = _rnd((16, 300), 1).cuda(), _rnd((16, 300), 2).cuda()
    opt, q = dlm.Muon([p], [g]), p.clone()
    torch.cuda.synchronize()
    assert dlm.load().dlm_muon_create(big, 1, 0, 0, C.byref(h)) == dlm.DLM_ENOMEM and h.value is None
    opt.step(0.1)
    q.add_(1.0)
    torch.cuda.synchronize()
    assert opt.status() == dlm.DLM_OK and bool(p.isfinite().all())


@pytest.mark.parametrize("shapes", [[(5, 16, 200), (3, 100, 30)], [(5, 9, 70), (3, 64, 100)], [(3, 20, 600), (2, 300, 64)],
                                    [(5, 16, 200), (3, 100, 30), (2, 50, 90)]])
def test_classes_in_joint_launches(shapes):
    """Tensors of several classes in one handle, whose launches hold waves for the widest: each class as by itself,
    bit for bit, a matrix that is not finite among them."""
    sides = []
    for groups in ([list(range(len(shapes)))], [[k] for k in range(len(shapes))]):
        ps = [_rnd(s, k, 0.02).cuda() for k, s in enumerate(shapes)]
        gs = [_rnd(s, 9 + k, 1e-3).cuda() for k, s in enumerate(shapes)]
        for g in gs:
            g[1, 0, 3] = float("nan")
        opts = [dlm.Muon([ps[k] for k in ks], [gs[k] for k in ks]) for ks in groups]
        for o in opts:
            o.step(0.1)
        assert all(o.status() == dlm.DLM_EDEVICE for o in opts)
        sides.append(ps + [m for o in opts for m in o.states])
    assert all(torch.equal(a, b) for a, b in zip(*sides))
    assert not torch.equal(sides[0][0][0].cpu(), _rnd(shapes[0], 0, 0.02)[0])


@pytest.mark.parametrize("shapes", [[(2, 16, 100)], [(2, 100, 30)], [(2, 60, 70)], [(2, 70, 90)], [(2, 16, 100), (2, 100, 30)],
                                    [(2, 16, 100), (2, 100, 60)]])
@pytest.mark.parametrize("steps", [1, 3])
def test_products_past_fp32(shapes, steps):
    """Coefficients whose products leave fp32's range leave the matrices, and set the error; up to 10^30 they do not."""
    for big in (False, True):
        a = (10.0 ** (60 if big else 30)) ** (1 / steps)
        ps = [_rnd(s, k, 0.02).cuda() for k, s in enumerate(shapes)]
        gs = [_rnd(s, 9 + k, 1e-3).cuda() for k, s in enumerate(shapes)]
        ms = [_rnd(s, 20 + k, 1e-3).cuda() for k, s in enumerate(shapes)]
        old = [t.clone() for t in ps + ms]
        opt = dlm.Muon(ps, gs, states=ms, steps=steps, coefs=(a, 0.0, 0.0), scale=1.0)
        opt.step(1e-30)
        assert opt.status() == (dlm.DLM_EDEVICE if big else dlm.DLM_OK)
        if big:
            assert all(torch.equal(x, y) for x, y in zip(old, ps + ms))
            continue
        for p, m, w in zip(ps, ms, old):
            u = BETA * m.double() + 0.05 * gs[[q is p for q in ps].index(True)].double()
            x = u / (u.flatten(1).norm(dim=1)[:, None, None] + EPS)
            # a's and the rate's roundings beside the product's
            ok = (p.double() - (w.double() - x)).abs() <= 16 * U * (w.double().abs() + x.abs()) + 1e-8 * x.abs().max()
            assert bool(ok.all())


def test_refusals_of_the_binding(monkeypatch):
    p, g = torch.zeros((4, 10), device="cuda"), torch.zeros((4, 10), device="cuda")
    for make in (lambda: dlm.Muon([], []), lambda: dlm.Muon([p], [g[:3]]), lambda: dlm.Muon([p], [g.cpu()]),
                 lambda: dlm.Muon([p.view(-1)], [g.view(-1)]), lambda: dlm.Muon([p], [g], weight_decay=[0.0, 0.0]),
                 lambda: dlm.Muon([p], [g], states=[torch.zeros(40, device="cuda")]), lambda: dlm.Muon([p.t()], [g.t()]),
                 lambda: dlm.Muon([p], [g], masters=[]), lambda: dlm.Muon([p], [g], scale="none"),
                 lambda: dlm.Muon([p], [g], steps=0), lambda: dlm.Muon([p], [g], steps=11),
                 lambda: dlm.Muon([p], [g], coefs=[(1, 1, 1)] * 4), lambda: dlm.Muon([p], [g], coefs=(1, 1))):
        with pytest.raises(ValueError):
            make()
    with pytest.raises(TypeError):
        dlm.Muon([p.half()], [g])
    for make in (lambda: dlm.Muon([p], [p]), lambda: dlm.Muon([p, p], [g, g]),
                 lambda: dlm.Muon([p], [g], masters=[torch.zeros((4, 10), device="cuda")]),
                 lambda: dlm.Muon([torch.zeros((513, 600), device="cuda")], [torch.zeros((513, 600), device="cuda")]),
                 lambda: dlm.Muon([p], [g], scale=float("nan"))):
        with pytest.raises(dlm.DLMError):
            make()
    opt = dlm.Muon([p], [g])
    with pytest.raises(dlm.DLMError):
        opt.step(float("nan"))
    with pytest.raises(ValueError):
        opt.step(1e-3, lr_scale=torch.zeros(2, device="cuda"))
    for bad in (dict(momentum=1.0), dict(eps=0.0), dict(coefs=(float("inf"), 1.0, 1.0))):
        with pytest.raises(dlm.DLMError):
            dlm.Muon([p], [g], **bad).step(1e-3)
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_cuda_getDevice", lambda: 1)
        for call in (lambda: opt.step(1e-3), opt.status):
            with pytest.raises(ValueError, match="current device"):
                call()
    empty = torch.zeros((0, 4, 10), device="cuda")
    e = dlm.Muon([empty, p], [empty.clone(), g])
    e.step(1.0)
    assert e.status() == dlm.DLM_OK and not p.any()
