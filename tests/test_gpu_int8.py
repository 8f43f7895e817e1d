"""The 8-bit products on the GPU against the plain form with exact sums.

Tolerances: codes and row scales are decided on exact quotients and have to be equal.  A result is a
whole number rounded to fp32 (U = 2^-24), times two fp32 factors: 3 U of itself; joined to another
value, U of the sum; bf16 rounds to half its eps."""
import pytest
import torch

import dynamic_lora_moe_amd as dlm
import int8_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _weight(o, i, seed):
    g = _gen(seed)
    return torch.randint(-127, 128, (o, i), generator=g).to(torch.int8), (torch.rand(o, generator=g) + 0.5) * 1e-3


def _x(T, d, dtype, seed, std=1.0):
    g = _gen(seed)
    return (torch.randn((T, d), generator=g) * torch.exp(torch.randn(d, generator=g)) * std).to(dtype)


def _near(got, want, dtype, extra=None):
    got, half = got.cpu().double(), torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
    tol = 3 * U * want.abs() + 2.0 ** -140
    if extra is not None:
        want = want + extra.double()
        tol = tol + U * want.abs()
    err = (got - want).abs()
    ok = (err <= tol + half * (want.abs() + tol)) | (got.isnan() & want.isnan())
    assert ok.all(), ((~ok).nonzero()[:4], got[~ok][:4], want[~ok][:4])


def _placed(t, shift):
    buf = torch.full((t.numel() + 64,), 3.0, dtype=t.dtype, device="cuda")
    v = buf[16 + shift:16 + shift + t.numel()].view(t.shape)
    v.copy_(t)
    return v, buf


def _guards(placed, shift):
    for v, buf in placed:
        assert (buf[:16 + shift] == 3).all() and (buf[16 + shift + v.numel():] == 3).all()


def _run(T, shapes, dtype, reads=None, back=True, accumulate=False, shift=0, rows=None, ws_fill=0x5A, stream=None):
    """shapes: (d_out, d_in) per problem; reads: which input each reads."""
    reads = reads or list(range(len(shapes)))
    placed, hx, hdx = [], {}, {}

    def put(t):
        placed.append(_placed(t, shift))
        return placed[-1][0]

    for k, r in enumerate(reads):
        if r not in hx:
            hx[r] = _x(T, shapes[k][1], dtype, 100 + r)
            hdx[r] = _x(T, shapes[k][1], dtype, 200 + r, 1e-3)
    x, dx = {r: put(t) for r, t in hx.items()}, {r: put(t) for r, t in hdx.items()}
    W, dy, y = [], [], []
    for k, (o, i) in enumerate(shapes):
        W.append(_weight(o, i, k))
        dy.append(_x(T, o, dtype, 300 + k, 1e-3))
        y.append(put(torch.full((T, o), 5.0, dtype=dtype)))
    dw = [(a.cuda(), b.cuda()) for a, b in W]
    grp = dlm.Int8Group([(x[r], a, b, yy) for r, (a, b), yy in zip(reads, dw, y)])
    for a, b in dw:  # the handle has its own
        a.zero_()
        b.zero_()
    n = T if rows is None else rows
    ws = grp.workspace(n).fill_(ws_fill)
    torch.cuda.synchronize()
    grp.run(T=rows, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for k, r in enumerate(reads):
        _near(y[k][:n], ref.forward(hx[r][:n], *W[k]), dtype)
        assert (y[k][n:] == 5).all()
    if back:
        ddy = [put(t) for t in dy]
        grp.bind_grads(ddy, [dx[r] for r in reads])
        wb = grp.backward_workspace(n).fill_(ws_fill)
        torch.cuda.synchronize()
        grp.backward(accumulate=accumulate, T=rows, workspace=wb, stream=stream)
        torch.cuda.synchronize()
        for r in hx:
            mine = [k for k in range(len(reads)) if reads[k] == r]
            want = ref.backward([dy[k][:n] for k in mine], [W[k][0] for k in mine], [W[k][1] for k in mine])
            _near(dx[r][:n], want, dtype, hdx[r][:n] if accumulate else None)
            assert torch.equal(dx[r][n:].cpu(), hdx[r][n:])
    for k, r in enumerate(reads):
        assert torch.equal(x[r].cpu(), hx[r])
    _guards(placed, shift)
    return y, dx


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 48, 64, 65, 100, 129, 300])
def test_rows(T, dtype):
    _run(T, [(72, 200), (16, 64), (130, 257)], dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("o,i", [(1, 1), (1, 300), (300, 1), (15, 63), (16, 64), (17, 65), (64, 128), (255, 129), (257, 1000), (8, 4096),
                                 (1001, 777), (520, 2056)])
def test_sizes(o, i, dtype):
    _run(5, [(o, i)], dtype)
    _run(140, [(o, i)], dtype, accumulate=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [3, 40, 200])
def test_shared_inputs(T, dtype):
    """Problems that share x and dx, of different widths, out of order, beside ones that do not."""
    _run(T, [(100, 96), (64, 72), (33, 96), (128, 96), (72, 72)], dtype, reads=[0, 1, 0, 0, 2])
    _run(T, [(100, 96), (64, 72), (33, 96), (128, 96), (72, 72)], dtype, reads=[0, 1, 0, 0, 2], accumulate=True)


@pytest.mark.parametrize("T,shapes", [(600, [(4096, 520)]), (1025, [(2048, 264), (264, 2048)]), (513, [(8192, 136)]),
                                      (2100, [(8190, 200)]), (2305, [(7000, 129), (640, 65), (100, 300)]), (4200, [(4100, 72)])])
def test_large_tiles(T, shapes):
    _run(T, shapes, torch.bfloat16)
    _run(T, shapes, torch.float32, accumulate=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 2, 3, 4])
def test_up_to_four_rows(T, dtype):
    """In one launch and in two (many columns, or codes that do not fit beside one another): each with a ragged
    end, a row of zeros and one that is not finite."""
    for o, i in ((300, 1000), (40000, 136), (64, 12300), (64, 70000), (33, 49000)):
        x, (W, ws) = _x(T, i, dtype, 1), _weight(o, i, 2)
        x[T - 1, 3] = float("nan") if T > 1 else 0.0
        x[0] = 0.0 if T > 2 else x[0]
        y = torch.empty((T, o), dtype=dtype, device="cuda")
        dlm.Int8Group([(x.cuda(), W.cuda(), ws.cuda(), y)]).run()
        _near(y, ref.forward(x, W, ws), dtype)
        alone = torch.empty((T, o), dtype=dtype, device="cuda")  # the rows among others: the same bits
        buf = torch.cat([x, _x(80, i, dtype, 3)]).cuda()
        many = torch.empty((T + 80, o), dtype=dtype, device="cuda")
        dlm.Int8Group([(buf, W.cuda(), ws.cuda(), many)]).run()
        alone.copy_(many[:T])
        assert torch.equal(alone.isnan(), y.isnan()) and torch.equal(alone.nan_to_num(), y.nan_to_num())


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("T", [7, 150])
def test_unaligned_buffers(T, shift):
    """Buffers at any multiple of their element's size: the same bits as aligned ones."""
    for dtype in (torch.float32, torch.bfloat16):
        a = _run(T, [(72, 200), (50, 61)], dtype, shift=shift)
        b = _run(T, [(72, 200), (50, 61)], dtype)
        assert all(torch.equal(p, q) for p, q in zip(a[0], b[0])) and all(torch.equal(a[1][r], b[1][r]) for r in a[1])


@pytest.mark.parametrize("rows", [0, 1, 70, 149])
def test_fewer_rows_than_the_buffers(rows):
    _run(150, [(72, 200), (50, 61)], torch.bfloat16, rows=rows)


def test_long_sums_stay_whole():
    """The longest sums of the largest codes, of one sign: 128 * 127 * 131072 in 32 bits."""
    d = 131072
    for T in (1, 65):
        x = torch.full((T, d), 3.0, device="cuda")
        W = torch.full((20, d), -128, dtype=torch.int8, device="cuda")
        W[1] = 127
        y = torch.empty((T, 20), device="cuda")
        grp = dlm.Int8Group([(x, W, torch.ones(20, device="cuda"), y)])
        grp.run()
        want = ref.product(torch.full((T, d), 127), torch.full((T,), 3.0) / 127, W.cpu(), None)
        _near(y, want, torch.float32)
    with pytest.raises(dlm.DLMError):
        dlm.Int8Group([(torch.zeros((1, d + 1), device="cuda"), torch.zeros((1, d + 1), dtype=torch.int8, device="cuda"),
                        torch.ones(1, device="cuda"), torch.zeros((1, 1), device="cuda"))])


def test_rows_that_are_not_finite_or_empty():
    """NaN and infinities give NaN in their own rows only; zeros give zeros; tiny and huge rows keep their codes."""
    for T in (12, 100):
        x, (W, ws) = _x(T, 100, torch.float32, 1), _weight(40, 100, 2)
        x[1, 5] = float("nan")
        x[2, 99] = float("inf")
        x[3] = 0.0
        x[4] *= 1e-36
        x[5] *= 1e30
        x[6, 1:] = 0.0
        x[7] = -x[7].abs().max()
        x[8] = torch.where(torch.arange(100) % 2 == 0, 1.0, 0.5)  # exact halves
        x[8, 1::4] *= -1
        x[9, 0] = -float("inf")
        y, dx, dy = torch.empty((T, 40), device="cuda"), torch.empty((T, 100), device="cuda"), _x(T, 40, torch.float32, 3, 1e-3)
        dy[1, 0], dy[2, 39], dy[3] = float("nan"), -float("inf"), 0.0
        dy[8] = torch.where(torch.arange(40) % 2 == 0, 1.0, 0.5) / ws.double()  # near halves after the channels' factors
        grp = dlm.Int8Group([(x.cuda(), W.cuda(), ws.cuda(), y)])
        grp.run()
        want = ref.forward(x, W, ws)
        assert want[1].isnan().all() and (want[3] == 0).all()
        _near(y, want, torch.float32)
        grp.bind_grads([dy.cuda()], [dx])
        grp.backward()
        _near(dx, ref.backward([dy], [W], [ws]), torch.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d", [(1, 1), (5, 16), (40, 100), (33, 4096), (3, 20000), (17, 8191)])
def test_codes(T, d, dtype):
    x = _x(T, d, dtype, d)
    x[0, : d // 2] = x[0, : d // 2] * 0.5
    q, s = dlm.quantize_rows(x.cuda())
    wq, wsc = ref.codes(x)
    assert torch.equal(q.cpu().long(), wq) and torch.equal(s.cpu(), wsc)
    buf = torch.full((T * d + 40,), 9, dtype=torch.int8, device="cuda")
    v = buf[17:17 + T * d].view(T, d)
    dlm.quantize_rows(x.cuda(), q=v)
    assert torch.equal(v, q)
    v.fill_(9)
    assert (buf == 9).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 4, 12, 64, 100, 700])
def test_rows_at_the_edge_of_fp32(T, dtype):
    """Rows up to the largest values of their type, with channels that bring the results back into range: finite."""
    o, i = 520, 136
    x, (W, ws) = _x(T, i, torch.float32, 1), _weight(o, i, 2)
    x = x / x.abs().amax(1, keepdim=True) * 3.3e38
    x[0, 1:], x[0, 0] = 0.0, 3.3e38
    x = x.to(dtype)
    ws = ws * 1e-3
    y = torch.empty((T, o), dtype=dtype, device="cuda")
    dlm.Int8Group([(x.cuda(), W.cuda(), ws.cuda(), y)]).run()
    want = ref.forward(x, W, ws)
    assert (want.abs() < 1e38).all() and (want.abs() > 1e34).any()
    _near(y, want, dtype)


def test_codes_of_every_half():
    """Rows whose quotients are exactly k + 1/2, and one fp32 step to either side."""
    h = torch.arange(0, 127, dtype=torch.float64) + 0.5
    for top in (127.0, 254.0, 63.5, 127 * 2.0 ** -20):
        mid = (h * (top / 127)).float()  # exact: top / 127 is a power of two
        rows = [torch.nextafter(mid, torch.zeros(())), mid, torch.nextafter(mid, torch.full((), 1e9))]
        x = torch.stack([torch.cat([r, -r, torch.tensor([top])]) for r in rows])
        q, _ = dlm.quantize_rows(x.cuda())
        assert torch.equal(q.cpu().long(), ref.codes(x)[0])
        assert torch.equal(q[1, :127].cpu().long(), torch.arange(127)) and torch.equal(q[2, :127].cpu().long(), torch.arange(1, 128))


def test_gradient_is_the_products_derivative():
    """With dy of whole codes (its rounding exact) dx is the derivative of the product of held weights: against
    differences of sum(dy * (x V)), V = w_scale W, linear in x."""
    T, o, i = 6, 24, 40
    W, _ = _weight(o, i, 1)
    ws = torch.full((o,), 2.0 ** -7)
    g = _gen(5)
    dy = torch.randint(-127, 128, (T, o), generator=g).float()
    dy[:, 0] = 127.0
    x, v = torch.randn((T, i), generator=g, dtype=torch.float64), torch.randn((T, i), generator=g, dtype=torch.float64)
    f = lambda s: ((x + s * v) @ (W.double() * ws.double()[:, None]).t() * dy).sum()  # noqa: E731
    dx = torch.empty((T, i), device="cuda")
    grp = dlm.Int8Group([(x.float().cuda(), W.cuda(), ws.cuda(), torch.empty((T, o), device="cuda"))])
    grp.bind_grads([dy.cuda()], [dx])
    grp.backward()
    want = f(0.5) - f(-0.5)
    assert abs(float((dx.cpu().double() * v).sum() - want)) <= 4 * U * float((dx.cpu().double() * v).abs().sum())


def test_unwanted_gradients_and_rebinding():
    T = 20
    x, y = torch.randn((T, 64), device="cuda"), [torch.empty((T, 32), device="cuda") for _ in range(3)]
    W = [_weight(32, 64, k) for k in range(3)]
    grp = dlm.Int8Group([(x, a.cuda(), b.cuda(), yy) for (a, b), yy in zip(W, y)])
    dy = [torch.randn((T, 32), generator=_gen(k)) for k in range(3)]
    dx = torch.full((T, 64), 7.0, device="cuda")
    with pytest.raises(dlm.DLMError):
        grp.backward()
    grp.bind_grads([None] * 3, [None] * 3)
    grp.backward()  # nothing is wanted
    grp.bind_grads([None, dy[1].cuda(), None], [None, dx, None])
    grp.backward()
    _near(dx, ref.backward(dy[1:2], [W[1][0]], [W[1][1]]), torch.float32)
    other = torch.empty_like(dx)
    grp.bind_grads([t.cuda() for t in dy], [other, None, other])
    grp.backward()
    _near(other, ref.backward([dy[0], dy[2]], [W[0][0], W[2][0]], [W[0][1], W[2][1]]), torch.float32)


def test_other_stream_and_own_workspace():
    s = torch.cuda.Stream()
    for T in (9, 200):
        a = _run(T, [(72, 200), (50, 61)], torch.bfloat16)
        b = _run(T, [(72, 200), (50, 61)], torch.bfloat16, stream=s, ws_fill=0xFF)
        assert all(torch.equal(p, q) for p, q in zip(a[0], b[0])) and all(torch.equal(a[1][r], b[1][r]) for r in a[1])
    x, (W, ws), y = _x(30, 64, torch.bfloat16, 1).cuda(), _weight(48, 64, 2), torch.empty((30, 48), dtype=torch.bfloat16, device="cuda")
    grp = dlm.Int8Group([(x, W.cuda(), ws.cuda(), y)])
    torch.cuda.synchronize()
    grp.run(stream=s)
    torch.cuda.synchronize()
    _near(y, ref.forward(x.cpu(), W, ws), torch.bfloat16)


def test_replayed_from_a_graph():
    """Replays on new inputs, with eager work between them, equal eager calls bit for bit."""
    for T in (2, 50, 300):
        x, (W, ws) = _x(T, 136, torch.bfloat16, 1).cuda(), _weight(72, 136, 2)
        y, dy, dx = (torch.zeros((T, n), dtype=torch.bfloat16, device="cuda") for n in (72, 72, 136))
        grp = dlm.Int8Group([(x, W.cuda(), ws.cuda(), y)])
        grp.bind_grads([dy], [dx])
        wf, wb = grp.workspace(T), grp.backward_workspace(T)

        def step():
            grp.run(workspace=wf)
            grp.backward(workspace=wb, accumulate=True)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for r in range(3):
            x.copy_(_x(T, 136, torch.bfloat16, 10 + r))
            dy.copy_(_x(T, 72, torch.bfloat16, 20 + r))
            dx.fill_(0.25)
            graph.replay()
            torch.cuda.synchronize()
            got = y.clone(), dx.clone()
            y.zero_()
            dx.fill_(0.25)
            step()
            torch.cuda.synchronize()
            assert torch.equal(got[0], y) and torch.equal(got[1], dx)


def test_past_2_32_elements():
    """More than 2^32 elements of x and of y: rows on both sides and at the end, as a small call gives them."""
    W, ws = _weight(8, 8192, 0)
    T = (1 << 32) // 8192 + 70
    print("int8", T, flush=True)
    x = torch.zeros((T, 8192), dtype=torch.bfloat16, device="cuda")
    tail = _x(130, 8192, torch.bfloat16, 1).cuda()
    x[-130:] = tail
    y = torch.empty((T, 8), dtype=torch.bfloat16, device="cuda")
    grp = dlm.Int8Group([(x, W.cuda(), ws.cuda(), y)])
    grp.run()
    _near(y[-130:], ref.forward(tail.cpu(), W, ws), torch.bfloat16)
    assert not y[:-130].any()
    dx = x  # the same in the other direction: x's memory is free now
    dy = torch.zeros((T, 8), dtype=torch.bfloat16, device="cuda")
    td = _x(130, 8, torch.bfloat16, 2).cuda()
    dy[-130:] = td
    grp.bind_grads([dy], [dx])
    grp.backward()
    _near(dx[-130:], ref.backward([td.cpu()], [W], [ws]), torch.bfloat16)
    assert not dx[:1000].any() and not dx[-1000:-130].any()


def test_refusals_of_the_binding(monkeypatch):
    x, (W, ws), y = torch.zeros((4, 32), device="cuda"), _weight(8, 32, 0), torch.zeros((4, 8), device="cuda")
    W, ws = W.cuda(), ws.cuda()
    for p in ([], [(x, W, ws, y[:3])], [(x, W.short(), ws, y)], [(x, W, ws.double(), y)], [(x, W.cpu(), ws, y)],
              [(x, W[:, :31].contiguous(), ws, y)], [(x.t(), W, ws, y)], [(x, W, ws, y.bfloat16())], [(x, W, ws[:7], y)]):
        with pytest.raises(ValueError):
            dlm.Int8Group(p)
    with pytest.raises(TypeError):
        dlm.Int8Group([(x.half(), W, ws, y.half())])
    grp = dlm.Int8Group([(x, W, ws, y)])
    for call in (lambda: grp.run(T=5), lambda: grp.run(T=-1), lambda: grp.bind_grads([], []),
                 lambda: grp.bind_grads([y[:3]], [x]), lambda: grp.bind_grads([y], [x.bfloat16()]),
                 lambda: dlm.quantize_rows(x[0]), lambda: dlm.quantize_rows(x, scale=torch.zeros(3, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(dlm.DLMError):
        grp.run(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    both = torch.zeros((8, 32), device="cuda")
    with pytest.raises(dlm.DLMError):  # y inside x
        dlm.Int8Group([(both[:4], W, ws, both.view(-1)[64:96].view(4, 8))]).run()
    with pytest.raises(dlm.DLMError):  # two problems write one y
        dlm.Int8Group([(x, W, ws, y), (x, W, ws, y)]).run()
    grp.bind_grads([y], [both[:4]])
    with pytest.raises(dlm.DLMError):
        dlm.Int8Group([(x, W, ws, y)]).backward()
    grp.bind_grads([both.view(-1)[:32].view(4, 8)], [both[:4]])
    with pytest.raises(dlm.DLMError):  # dy inside dx
        grp.backward()
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_cuda_getDevice", lambda: 1)
        for call in (grp.run, grp.backward, lambda: dlm.quantize_rows(x)):
            with pytest.raises(ValueError, match="current device"):
                call()
