"""AdamW over many tensors on the GPU against the plain binary64 form.

Tolerances (u = 2^-24).  One step from the same state.
  m: fp32 betas, two products and a sum: 4 u (|b1 m| + |(1 - b1) g|); v the same.
  w: the decay factor, a product, the step's product and the difference: 4 u |w|,
     and lr times the step's own error: 16 u of it (two corrections, square
     root, sum, quotient, product, each at most u, the corrections' factors 2 u)
     and what m's and v's errors make of it.
  p: bf16 rounding of w, half of eps: 2^-8 |w|.
8-bit codes and scales have to be equal: both sides are binary64 there."""
import numpy as np
import pytest
import torch

import adamw_ref as ref
import dynamic_lora_moe_amd as dlm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
B1, B2, EPS = 0.9, 0.999, 1e-8
SIZES = [1, 3, 255, 256, 257, 4095, 4096, 4097, 0, 10001, 70000]


def _rnd(n, seed, std=1.0):
    return torch.randn(n, generator=torch.Generator().manual_seed(seed)) * std


def _f64(t):
    return t.detach().cpu().double().numpy()


def _place(t, shift):
    """t on the device, `shift` elements behind an aligned address, with a guard on both sides."""
    buf = torch.full((t.numel() + 64,), 3, dtype=t.dtype, device="cuda")
    v = buf[16 + shift:16 + shift + t.numel()]
    v.copy_(t)
    return v, buf


def _make(sizes, p_dtype, g_dtype, master, bits, seed, shift=0):
    ps, gs, ws, st, bufs = [], [], [], [], []
    put = lambda t: [bufs.append((v := _place(t, shift)) + (t.numel(),)), v[0]][1]  # noqa: E731
    for k, n in enumerate(sizes):
        w = _rnd(n, seed + k, 0.02)
        ps.append(put(w.to(p_dtype)))
        gs.append(put(_rnd(n, seed + 100 + k, 1e-3).to(g_dtype)))
        ws.append(put(w) if master else None)
        if bits == 32:
            st.append((put(_rnd(n, seed + 200 + k, 3e-4)), put(_rnd(n, seed + 300 + k, 1e-3).square())))
        else:
            nb = -(-n // 256)
            gen = torch.Generator().manual_seed(seed + 400 + k)
            st.append((put(torch.randint(-127, 128, (n,), generator=gen).to(torch.int8)),
                       put(torch.randint(0, 256, (n,), generator=gen).to(torch.uint8)),
                       put(torch.rand(nb, generator=gen) * 1e-3), put(torch.rand(nb, generator=gen) * 1e-6)))
    return ps, gs, ws, st, bufs, shift


def _guards(bufs, shift):
    for v, buf, n in bufs:
        assert (buf[:16 + shift] == 3).all() and (buf[16 + shift + n:] == 3).all()


def _run(sizes, p_dtype, g_dtype, master, bits, steps=3, shift=0, step0=0, seed=1):
    ps, gs, ws, st, bufs, shift = _make(sizes, p_dtype, g_dtype, master, bits, seed, shift)
    wd = [0.01 * (k % 3) for k in range(len(sizes))]
    opt = dlm.AdamW(ps, gs, masters=ws, state_bits=bits, states=st, weight_decay=wd, step=step0, seed=5)
    for i in range(steps):
        snap = [(p.clone(), None if w is None else w.clone(), tuple(x.clone() for x in s)) for p, w, s in zip(ps, ws, st)]
        opt.step(1e-3)
        torch.cuda.synchronize()
        for k in range(len(sizes)):
            _compare(k, snap[k], ps[k], gs[k], ws[k], st[k], bits, step0 + i + 1, 1e-3, wd[k])
        for g in gs:
            g.mul_(-0.5)
    _guards(bufs, shift)
    assert opt.status() == (step0 + steps, dlm.DLM_OK)
    return ps, st


def _compare(k, snap, p, gr, w_new, st, bits, t, lr, wd, gscale=1.0):
    p0, w0, s0 = snap
    if not p0.numel():
        return
    g = (gr.float() * gscale).cpu().double().numpy()
    m0, v0 = (_f64(s0[0]), _f64(s0[1])) if bits == 32 else ref.decode(*[x.cpu().numpy() for x in s0])
    m, v = ref.moments(g, m0, v0, B1, B2)
    em = 4 * U * (np.abs(B1 * m0) + np.abs((1 - B1) * g))
    ev = 4 * U * (B2 * v0 + (1 - B2) * g * g) + 2.0 ** -148
    if bits == 32:
        assert (np.abs(_f64(st[0]) - m) <= em + 2.0 ** -149).all()
        assert (np.abs(_f64(st[1]) - v) <= ev).all()
    else:
        for x, y in zip(st, ref.encode(m, v, 5, t, k)):
            assert np.array_equal(x.cpu().numpy(), y), (k, x.dtype)
    w = _f64(p0 if w0 is None else w0)
    new, s = ref.update(w, m, v, t, lr, B1, B2, EPS, wd)
    es = 16 * U * np.abs(s) + np.abs(s) * ev / np.maximum(v, 1e-300) + em / (1 - B1 ** t) / (np.sqrt(v / (1 - B2 ** t)) + EPS)
    ew = 4 * U * np.abs(w) + lr * es
    if w0 is not None:
        assert (np.abs(_f64(w_new) - new) <= ew).all()
        assert torch.equal(p, w_new.to(p.dtype))
    else:
        half = torch.finfo(p.dtype).eps / 2 if p.dtype != torch.float32 else 0.0
        assert (np.abs(_f64(p) - new) <= ew + half * (np.abs(new) + ew)).all()


TYPES = [(torch.float32, torch.float32, False), (torch.bfloat16, torch.float32, True), (torch.bfloat16, torch.bfloat16, True),
         (torch.bfloat16, torch.bfloat16, False), (torch.float32, torch.bfloat16, False)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dtype,g_dtype,master", TYPES)
def test_sizes_and_types(bits, p_dtype, g_dtype, master):
    _run(SIZES, p_dtype, g_dtype, master, bits)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_unaligned_tensors(bits, shift):
    """Tensors at any multiple of their element's size: the same results as aligned ones, bit for bit."""
    a, sa = _run([4097, 300, 5], torch.bfloat16, torch.float32, True, bits, shift=shift)
    b, sb = _run([4097, 300, 5], torch.bfloat16, torch.float32, True, bits, shift=0)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    for x, y in zip(sa, sb):
        assert all(torch.equal(q, r) for q, r in zip(x, y))


@pytest.mark.parametrize("bits", [32, 8])
def test_from_zero_moments_and_resumed(bits):
    """Fresh moments; then a second handle that goes on from the first one's state, against one that ran through."""
    n = 5000
    w = _rnd(n, 1, 0.02).cuda()
    g = _rnd(n, 2).cuda()
    one, two = w.clone(), w.clone()
    a = dlm.AdamW([one], [g], state_bits=bits, seed=9)
    for _ in range(6):
        a.step(1e-2)
    b = dlm.AdamW([two], [g], state_bits=bits, seed=9)
    for _ in range(3):
        b.step(1e-2)
    assert b.status() == (3, dlm.DLM_OK)
    c = dlm.AdamW([two], [g], state_bits=bits, states=b.states, seed=9, step=3)
    for _ in range(3):
        c.step(1e-2)
    torch.cuda.synchronize()
    assert torch.equal(one, two)
    # a constant gradient: every step goes lr against its sign, but for rounding
    # of the moments (none enters the step that made them) and the decay
    m, v = a.read_state(0)
    assert torch.isfinite(m).all() and (v >= 0).all()
    if bits == 32:
        assert (one - (w - 6e-2 * torch.sign(g))).abs().max() <= 6 * (1e-2 * 1e-2 * 0.2 + 1e-2 * 1e-3)


def test_8bit_blocks_at_the_edges():
    """Blocks of zeros, of one element, of equal, huge, tiny and denormal values."""
    n = 256 * 9 + 17
    g = torch.zeros(n)
    g[256] = 1e-3
    g[512:768] = 1.0
    g[768:1024] = _rnd(256, 1) * 1e15
    g[1024:1280] = _rnd(256, 2) * 1e-18
    g[1280:1536] = _rnd(256, 3) * 1e-30   # v below fp32's range: its scale and codes are 0
    g[1536:1792] = 2.0 ** -torch.arange(256).float().clamp(max=120)
    g[1792:2048] = -(10.0 ** -(torch.arange(256).float() / 40))
    g[2048] = -1e-40
    g[n - 1] = 5.0
    gd = g.cuda()
    p = torch.zeros(n, device="cuda")
    opt = dlm.AdamW([p], [gd], state_bits=8, weight_decay=0.0, seed=5)
    for t in (1, 2, 3):
        snap = (p.clone(), None, tuple(x.clone() for x in opt.states[0]))
        opt.step(1e-3)
        torch.cuda.synchronize()
        m0, v0 = ref.decode(*[x.cpu().numpy() for x in snap[2]])
        m, v = ref.moments(_f64(gd), m0, v0, B1, B2)
        for x, y in zip(opt.states[0], ref.encode(m, v, 5, t, 0)):
            assert np.array_equal(x.cpu().numpy(), y)
        mo, vo = opt.read_state(0)
        rm, rv = ref.decode(*[x.cpu().numpy() for x in opt.states[0]])
        assert np.array_equal(mo.cpu().numpy(), rm.astype(np.float32)) or np.abs(_f64(mo) - rm).max() <= U * np.abs(rm).max()
        assert (np.abs(_f64(vo) - rv) <= U * rv + 2.0 ** -149).all()
    assert torch.isfinite(p).all()
    assert (p[:256] == 0).all() and p[256] < 0


def test_8bit_rounding_is_unbiased_and_moves():
    """The stored moments' mean is the exact one: N elements of one value, whose stored values are two
    neighbouring codes, so their mean is off by at most 5 standard deviations, each at most half the
    codes' distance / sqrt(N), and by the noise's own grain, 2^-17 of the distance."""
    n = 256 * 400
    g = torch.zeros(n)
    g[::256] = 1.0  # each block's scales
    rest = torch.arange(n) % 256 != 0
    g[rest] = 0.2345
    p = torch.zeros(n, device="cuda")
    opt = dlm.AdamW([p], [g.cuda()], state_bits=8, seed=3)
    opt.step(1e-3)
    m, v = opt.read_state(0)
    for x, exact, codes, power in ((m, (1 - B1) * 0.2345, 127, 2), (v, (1 - B2) * 0.2345 ** 2, 255, 4)):
        top = {2: 1 - B1, 4: 1 - B2}[power]
        x = _f64(x)[rest.numpy()]
        c = np.floor(codes * (exact / top) ** (1 / power))
        dist = top * ((c + 1) ** power - c ** power) / codes ** power
        assert len(np.unique(x)) == 2
        # (the fp32 gradient and scale put the exact value 2^-23 off)
        assert abs(x.mean() - exact) <= 5 * dist / 2 / np.sqrt(len(x)) + dist * 2.0 ** -17 + exact * 2.0 ** -22


def test_8bit_second_moment_decays():
    """With no gradient v falls by b2 a step in the mean, though a step is far less than a code.  One
    element a block has the gradient that holds its v, and so the scale.  After 500 steps the mean of N
    stored values is within 6 standard deviations: each step adds a variance of at most (distance / 2)^2,
    the distance at most 2% of the start (between fourth powers at codes of 203 to 230: 4 / 203), and
    the noise's grain 2^-17 of it."""
    blocks, steps = 64, 500
    n = 256 * blocks
    code = torch.full((n,), 230, dtype=torch.uint8)
    g = torch.zeros(n)
    code[::256], g[::256] = 255, 1e-2
    st = [(torch.zeros(n, dtype=torch.int8, device="cuda"), code.cuda(), torch.zeros(blocks, device="cuda"),
           torch.full((blocks,), 1e-4, device="cuda"))]
    start = 1e-4 * (230 / 255) ** 4
    opt = dlm.AdamW([torch.zeros(n, device="cuda")], [g.cuda()], state_bits=8, states=st, step=1000)
    for _ in range(steps):
        opt.step(1e-3)
    _, v = opt.read_state(0)
    v = _f64(v)[np.arange(n) % 256 != 0]
    exact = start * B2 ** steps
    sd = 0.02 / 2 * start * np.sqrt(steps) / np.sqrt(len(v))
    assert abs(v.mean() - exact) <= 6 * sd + steps * 0.02 * start * 2.0 ** -17
    assert opt.status()[0] == 1000 + steps


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_gradients_that_are_not_finite(bits, value):
    """The element (with 8 bits its block) stays as it was, the others take their step, the error is reported once."""
    n = 1000
    ps, gs, ws, st, _, _ = _make([n, 300], torch.float32, torch.float32, False, bits, 7)
    gs[0][600] = value
    opt = dlm.AdamW(ps, gs, state_bits=bits, states=st, seed=5)
    snap = [(p.clone(), tuple(x.clone() for x in s)) for p, s in zip(ps, st)]
    opt.step(1e-3)
    torch.cuda.synchronize()
    assert opt.status() == (1, dlm.DLM_EDEVICE) and opt.status() == (1, dlm.DLM_OK)
    skip = torch.zeros(n, dtype=torch.bool, device="cuda")
    skip[600 if bits == 32 else slice(512, 768)] = True
    moved = ps[0] != snap[0][0]
    assert not moved[skip].any() and moved[~skip].float().mean() > 0.95
    for x, y in zip(st[0][:2], snap[0][1][:2]):
        assert torch.equal(x[skip], y[skip])
    assert torch.isfinite(ps[0]).all()
    gs[0][600] = 0.0
    opt.step(1e-3)
    assert opt.status() == (2, dlm.DLM_OK)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value,taken", [(1e19, True), (-1e20, True), (5.8e20, True), (5.9e20, False), (-1e21, False)])
def test_the_largest_gradients(bits, value, taken):
    """Both widths take a gradient as long as the new v is finite in fp32, here up to 5.83e20."""
    ps, gs, ws, st, _, _ = _make([1000, 300], torch.float32, torch.float32, False, bits, 7)
    gs[0][600] = value
    opt = dlm.AdamW(ps, gs, state_bits=bits, states=st, weight_decay=0.0, seed=5)
    p0, s0 = ps[0].clone(), tuple(x.clone() for x in st[0])
    opt.step(1e-3)
    torch.cuda.synchronize()
    assert opt.status() == (1, dlm.DLM_OK if taken else dlm.DLM_EDEVICE)
    if not taken:
        assert ps[0][600] == p0[600] and all(x[600] == y[600] for x, y in zip(st[0][:2], s0))
        return
    m0, v0 = (_f64(s0[0]), _f64(s0[1])) if bits == 32 else ref.decode(*[x.cpu().numpy() for x in s0])
    m, v = ref.moments(_f64(gs[0]), m0, v0, B1, B2)
    if bits == 8:
        for x, y in zip(st[0], ref.encode(m, v, 5, 1, 0)):
            assert np.array_equal(x.cpu().numpy(), y)
    else:  # (two products and a sum for v, r2 rounded: 4 u; the old moments are nothing beside it)
        assert abs(float(st[0][0][600]) - m[600]) <= 4 * U * abs(m[600])
        assert abs(float(st[0][1][600]) - v[600]) <= 4 * U * v[600]
    new, s = ref.update(_f64(p0), m, v, 1, 1e-3, B1, B2, EPS, 0.0)
    # the step's sixteen roundings and what 4 u of m and of v (a root of it) make of it
    assert abs(float(ps[0][600]) - new[600]) <= 4 * U * abs(float(p0[600])) + 1e-3 * (16 + 4 + 2) * U * abs(s[600])


@pytest.mark.parametrize("value", [1e15, 1e20, 5e20])
def test_8bit_neighbours_of_a_huge_gradient(value):
    """One huge gradient in a block: the others' codes go to the bottom of its range, their steps do not."""
    ps, gs, ws, st, _, _ = _make([1000], torch.float32, torch.float32, False, 8, 7)
    st[0][1][512:768] = 0
    gs[0][512:600] = torch.logspace(-3, -18, 88)
    gs[0][600] = value
    opt = dlm.AdamW(ps, gs, state_bits=8, states=st, weight_decay=0.0, seed=5)
    p0, s0 = ps[0].clone(), tuple(x.clone() for x in st[0])
    opt.step(1e-3)
    torch.cuda.synchronize()
    assert opt.status() == (1, dlm.DLM_OK)
    _compare(0, (p0, None, s0), ps[0], gs[0], None, st[0], 8, 1, 1e-3, 0.0)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-45, 1e-40, 2.0 ** -126, 1e-30])
def test_the_least_eps(bits, eps):
    """Elements without a gradient stay where they are at any eps that is taken; the 8-bit step refuses those below 2^-126."""
    p = torch.full((600,), 0.5, device="cuda")
    g = torch.zeros(600, device="cuda")
    g[:100] = 1e-3
    opt = dlm.AdamW([p], [g], state_bits=bits, eps=eps, weight_decay=0.0)
    if bits == 8 and eps < 2.0 ** -126:
        with pytest.raises(dlm.DLMError, match="eps"):
            opt.step(1e-3)
        assert opt.status() == (0, dlm.DLM_OK)
        return
    opt.step(1e-3)
    torch.cuda.synchronize()
    assert (p[100:] == 0.5).all() and (p[:100] < 0.5).all() and torch.isfinite(p).all()


def test_the_count_goes_on_past_31_bits():
    p, g = torch.zeros(10, device="cuda"), torch.ones(10, device="cuda")
    opt = dlm.AdamW([p], [g], step=(1 << 31) - 1)
    for k in range(3):
        opt.step(1e-3)
        assert opt.status() == ((1 << 31) + k, dlm.DLM_OK)


def test_scales_on_the_device():
    """lr_scale and grad_scale multiply as the arguments would."""
    n = 3000
    w, g = _rnd(n, 1, 0.02).cuda(), _rnd(n, 2, 1e-3).cuda()
    a, b = w.clone(), w.clone()
    half = torch.tensor([0.5], device="cuda")
    x, y = dlm.AdamW([a], [g]), dlm.AdamW([b], [g * 0.5])
    for _ in range(3):
        x.step(2e-3, lr_scale=half, grad_scale=half)
        y.step(1e-3)
    assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_counts_on_replay(bits):
    """Three replays, with eager work and synchronisation between them, equal three eager steps, bit for bit."""
    n = 9000
    w, g = _rnd(n, 1, 0.02), _rnd(n, 2, 1e-3).cuda()
    a, b = w.cuda(), w.cuda()
    x = dlm.AdamW([a], [g], state_bits=bits, seed=4)
    y = dlm.AdamW([b], [g], state_bits=bits, seed=4)
    lr = torch.tensor([1.0], device="cuda")
    x.step(1e-3, lr_scale=lr)
    y.step(1e-3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.step(1e-3, lr_scale=lr)
    for k in range(3):
        lr.fill_(1.0 / (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        y.step(1e-3, lr_scale=lr)
        torch.cuda.synchronize()
        assert torch.equal(a, b)
    assert x.status() == (4, dlm.DLM_OK)
    assert all(torch.equal(p, q) for p, q in zip(x.states[0], y.states[0]))


def test_other_stream_and_many_tensors():
    """Two hundred tensors on a stream of their own, against the same on the current one."""
    sizes = [(37 * k) % 6000 + 1 for k in range(200)]
    out = []
    for stream in (None, torch.cuda.Stream()):
        ps = [_rnd(n, k, 0.02).cuda() for k, n in enumerate(sizes)]
        gs = [_rnd(n, 500 + k, 1e-3).cuda() for k, n in enumerate(sizes)]
        opt = dlm.AdamW(ps, gs, state_bits=8, seed=2)
        torch.cuda.synchronize()
        opt.step(1e-3, stream=stream)
        torch.cuda.synchronize()
        out.append(ps)
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_calls_with_another_device_current(monkeypatch):
    """A stream of another device orders nothing here: step() and status() refuse the call."""
    opt = dlm.AdamW([torch.zeros(10, device="cuda")], [torch.ones(10, device="cuda")])
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_cuda_getDevice", lambda: 1)
        for call in (lambda: opt.step(1e-3), opt.status):
            with pytest.raises(ValueError, match="current device"):
                call()
    assert opt.status() == (0, dlm.DLM_OK)


@pytest.mark.parametrize("n,shift", [(1, 0), (2, 1), (255, 1), (256, 0), (1000, 0), (1001, 3), (70001, 2), (70001, 0), (70004, 0)])
def test_read_back_of_every_element(n, shift):
    """Codes of every kind with scales from 1e-40 to 1e20 beside one another, sizes and places that end inside
    four elements: each value to one fp32 rounding of its own, on guarded outputs too."""
    gen = torch.Generator().manual_seed(n + shift)
    nb = -(-n // 256)
    put = lambda t: _place(t, shift)[0]  # noqa: E731
    st = (put(torch.randint(-127, 128, (n,), generator=gen).to(torch.int8)),
          put(torch.randint(0, 256, (n,), generator=gen).to(torch.uint8)),
          put(10.0 ** (torch.rand(nb, generator=gen) * 60 - 40)), put(10.0 ** (torch.rand(nb, generator=gen) * 60 - 40)))
    rm, rv = ref.decode(*[x.cpu().numpy() for x in st])
    outs = [_place(torch.zeros(n), shift) for _ in range(2)]
    for mo, vo in (dlm.adamw_read_state(*st), dlm.adamw_read_state(*st, m_out=outs[0][0], v_out=outs[1][0])):
        assert (np.abs(_f64(mo) - rm) <= U * np.abs(rm) + 2.0 ** -149).all()
        assert (np.abs(_f64(vo) - rv) <= U * rv + 2.0 ** -149).all()
    for v, buf in outs:
        assert (buf[:16 + shift] == 3).all() and (buf[16 + shift + n:] == 3).all()


def test_moments_read_back_after_steps_element_by_element():
    """What steps over blocks from 1e15 down to 1e-18 leave, read back: m and v each to one rounding."""
    n = 256 * 5 + 3
    g = torch.cat([_rnd(256, k) * 10.0 ** e for k, e in enumerate((15, 3, 0, -8, -18))] + [torch.tensor([-1.0, 0.0, 2e-5])])
    opt = dlm.AdamW([torch.zeros(n, device="cuda")], [g.cuda()], state_bits=8, seed=5)
    for _ in range(3):
        opt.step(1e-3)
        mo, vo = opt.read_state(0)
        rm, rv = ref.decode(*[x.cpu().numpy() for x in opt.states[0]])
        assert (np.abs(_f64(mo) - rm) <= U * np.abs(rm) + 2.0 ** -149).all()
        assert (np.abs(_f64(vo) - rv) <= U * rv + 2.0 ** -149).all()
        assert (np.sign(rm) == np.sign(g.double().numpy()))[rm != 0].all() and (rm != 0).mean() > 0.9


def test_refusals_of_the_binding():
    p, g = torch.zeros(10, device="cuda"), torch.zeros(10, device="cuda")
    with pytest.raises(ValueError):
        dlm.AdamW([], [])
    with pytest.raises(ValueError):
        dlm.AdamW([p], [g[:9]])
    with pytest.raises(ValueError):
        dlm.AdamW([p], [g.cpu()])
    with pytest.raises(ValueError):
        dlm.AdamW([p], [g], state_bits=16)
    with pytest.raises(ValueError):
        dlm.AdamW([p], [g], weight_decay=[0.0, 0.0])
    with pytest.raises(ValueError):
        dlm.AdamW([p], [g], states=[(torch.zeros(10, device="cuda"), torch.zeros(9, device="cuda"))])
    with pytest.raises(ValueError):
        dlm.AdamW([p.view(2, 5).t()], [g.view(2, 5).t()])
    with pytest.raises(TypeError):
        dlm.AdamW([p.half()], [g])
    with pytest.raises(dlm.DLMError):
        dlm.AdamW([p], [p])
    with pytest.raises(dlm.DLMError):
        dlm.AdamW([p, p], [g, g])
    with pytest.raises(dlm.DLMError):
        dlm.AdamW([p], [g], masters=[torch.zeros(10, device="cuda")])
    opt = dlm.AdamW([p], [g])
    with pytest.raises(dlm.DLMError):
        opt.step(float("nan"))
    with pytest.raises(ValueError):
        opt.step(1e-3, lr_scale=torch.zeros(2, device="cuda"))
    bad = dlm.AdamW([p], [g], beta2=1.0)
    with pytest.raises(dlm.DLMError):
        bad.step(1e-3)
