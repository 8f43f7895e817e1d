"""The balance loss, its counts and its gradient on the GPU against the plain binary64 form.

Tolerances: an fp32 p is off by `relative` of itself (balance_ref, which counts its roundings);
a mean adds up to eight rows in fp32 (a workgroup's rounds) and rounds once: 9 of 2^-24 more.
What lies below 2^-126 of a row's largest is 0 in fp32.  bf16 rounds a gradient to half its eps.
Counts and rows are whole numbers and have to be equal."""
import math

import pytest
import torch

import balance_ref as ref
import dynamic_lora_moe_amd as dlm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
INF = float("inf")


def _inputs(T, E, k, dtype, seed, masked=0.0, pad=0, spread=2.0, shift=0.0):
    gen = torch.Generator().manual_seed(seed)
    l = torch.randn((T, E), generator=gen) * spread + torch.randn(E, generator=gen) + shift
    if masked:
        l = l.masked_fill(torch.rand((T, E), generator=gen) < masked, -INF)
    if pad:
        l[max(T - pad, 0):] = -INF
    l = l.to(dtype)
    key = l.float() + torch.randn((T, E), generator=gen) * 0.1
    top = key.topk(k, 1)
    return l, torch.where(top.values > -INF, top.indices, -1).int()


def _check(l, idx, score, alpha, zeta, offsets, dev_logits=None, add=None, dloss=None):
    T, E = l.shape
    k = idx.shape[1]
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x = l.cuda() if dev_logits is None else dev_logits
    loss, counts, rows, probs = dlm.balance(x, idx.cuda(), score=score, alpha=alpha, zeta=zeta, offsets=off)
    wl, wc, wr, wp = ref.balance(l, idx, score, alpha, zeta, offsets)
    assert torch.equal(counts.cpu().long(), wc) and torch.equal(rows.cpu().long(), wr)
    p, _, lse, _, live = ref.scores(l.double(), score)
    b = ref.borders(T, offsets)
    rel = ref.relative(l.double(), p, score)
    S = len(b) - 1
    tl = torch.zeros(2, dtype=torch.float64)
    for q in range(S):
        cut, n = slice(b[q], b[q + 1]), max(int(wr[q]), 1)
        tp = ((rel[cut] + 9 * U) * p[cut]).sum(0) / n + 2.0 ** -120
        assert (probs[q].cpu().double() - wp[q]).abs().le(tp).all(), q
        tl[0] += abs(alpha) / S * (E / (k * n) * wc[q] * tp).sum()
        # the log sum: its exponentials' error, the logarithm (2^-22 of 40 at most) and two roundings
        el = 2.0 ** -22 * 8 + 3 * U * lse[cut].abs() + 64 * U
        tl[1] += abs(zeta) / S / n * (2 * lse[cut].abs() * el + el * el).sum()
    assert (loss.cpu().double() - wl).abs().le(tl + U * wl.abs()).all(), (loss, wl, tl)
    out = None if add is None else add.clone().cuda()
    if out is None and offsets is not None:
        out = torch.full_like(x, 7.0)
    dd = None if dloss is None else torch.tensor(dloss, device="cuda")
    dl = dlm.balance_backward(x, counts, rows, k, score=score, alpha=alpha, zeta=zeta, offsets=off, dlogits=out, dloss=dd,
                              accumulate=add is not None)
    want, tol = ref.backward(l, wc, wr, k, score, alpha, zeta, offsets, dloss or (1.0, 1.0))
    got = dl.cpu().double()
    half = torch.finfo(l.dtype).eps / 2
    base = 0 if add is None else add.double()
    want = want + base
    inside = slice(b[0], b[-1])
    bad = (got[inside] - want[inside]).abs() > tol[inside] + half * (want[inside].abs() + tol[inside]) + 2.0 ** -120
    assert not bad.any(), (bad.nonzero()[:4], got[inside][bad][:4], want[inside][bad][:4], tol[inside][bad][:4])
    for rows_out in (slice(0, b[0]), slice(b[-1], T)):  # rows of no sequence: as they were
        assert (got[rows_out] == (7.0 if add is None else add[rows_out].double())).all()
    return loss, counts, rows, probs, dl


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 2, 1), (64, 8, 2), (257, 16, 2), (130, 17, 3), (70, 31, 4), (513, 60, 6),
                                   (300, 64, 8), (99, 100, 5), (257, 128, 8), (65, 255, 16), (200, 256, 8), (37, 300, 7),
                                   (129, 512, 8)])
def test_sizes(T, E, k, score, dtype):
    l, idx = _inputs(T, E, k, dtype, T + E)
    _check(l, idx, score, 0.01, 1e-3 if score == "softmax" else 0.0, None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("offsets", [[0, 400], [0, 0, 0, 400, 400], [0, 1, 2, 3, 64, 65, 128, 300, 390], [5, 130, 131, 397],
                                     [400, 400, 400], list(range(0, 401)), [0] * 9 + [400], [7, 7]])
def test_sequences(offsets, score, dtype):
    """Packed sequences: borders inside and on blocks, empty ones, one row each, rows before and behind them."""
    l, idx = _inputs(400, 60, 4, dtype, len(offsets), masked=0.1, pad=20)
    _check(l, idx, score, 0.5, 0.1 if score == "softmax" else 0.0, offsets)
    add = torch.randn((400, 60), generator=torch.Generator().manual_seed(9)).mul(1e-3).to(dtype)
    _check(l, idx, score, 0.5, 0.1 if score == "softmax" else 0.0, offsets, add=add, dloss=[2.0, -0.5])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks_and_odd_values(score):
    """Rows that leave one expert or none, NaN and infinities, the lowest value, far logits, repeated and bad slots."""
    l, idx = _inputs(40, 12, 3, torch.float32, 3)
    l[0] = -INF
    l[1, 1:] = -INF
    l[2] = float("nan")
    l[3, ::2] = float("nan")
    l[4, 5] = INF
    l[5] = torch.finfo(torch.float32).min
    l[6] = -1000.0 + torch.arange(12)
    l[7] = 1000.0 - torch.arange(12)
    l[8] = torch.linspace(-200, 200, 12)
    l[9] = -45.0 + torch.arange(12)
    l[10] = -1e30
    l[11, :4] = -0.0
    idx[12] = torch.tensor([4, 4, 4])
    idx[13] = torch.tensor([-1, 12, 2 ** 31 - 1])
    idx[14] = torch.tensor([-2 ** 31, 0, 11])
    idx[3] = torch.tensor([0, 1, 2])  # two of them not available
    idx[0] = torch.tensor([1, 2, 3])  # none
    z = 1e-3 if score == "softmax" else 0.0
    keep = [t for t in range(40) if t != 4 and t not in (5, 10)]
    _check(l[keep], idx[keep], score, 0.1, z, None)
    # far from what fp32 squares: the balance term alone
    _check(l, idx, score, 0.1, 0.0, [0, 3, 6, 11, 40])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_pitch_and_alignment(dtype):
    """Rows a pitch apart, and buffers at odd elements: the same bits as packed ones."""
    l, idx = _inputs(90, 24, 2, dtype, 5)
    _, counts, rows, probs, dl = _check(l, idx, "softmax", 0.1, 0.01, None)
    for pitch, shift in ((32, 0), (29, 3), (24, 1)):
        buf = torch.full((90 * pitch + 8,), 5.0, dtype=dtype, device="cuda")
        view = buf[shift:shift + 90 * pitch].view(90, pitch)[:, :24]
        view.copy_(l)
        res = dlm.balance(view, idx.cuda(), alpha=0.1, zeta=0.01)
        assert torch.equal(res[1], counts) and torch.equal(res[2], rows) and torch.equal(res[3], probs)
        out = torch.full((90 * pitch + 8,), 5.0, dtype=dtype, device="cuda")
        ov = out[shift:shift + 90 * pitch].view(90, pitch)[:, :24]
        dlm.balance_backward(view, counts, rows, 2, alpha=0.1, zeta=0.01, dlogits=ov)
        assert torch.equal(ov, dl)
        ov.fill_(5.0)
        assert (out == 5.0).all()  # nothing beside the rows


def test_as_many_sequences_as_there_may_be():
    T, S = 70000, dlm.MAX_BALANCE_SEQS
    l, idx = _inputs(T, 8, 2, torch.float32, 6)
    cut = torch.randint(0, T + 1, (S - 1,), generator=torch.Generator().manual_seed(1)).sort().values
    off = torch.cat([torch.zeros(1, dtype=torch.long), cut, torch.tensor([T])]).int()
    loss, counts, rows, probs = dlm.balance(l.cuda(), idx.cuda(), alpha=1.0, offsets=off.cuda())
    n = off.diff().long()
    seq = torch.repeat_interleave(torch.arange(S), n)
    p = ref.scores(l.double(), "softmax")[0]
    want = torch.zeros((S, 8), dtype=torch.float64).index_add_(0, seq, p) / n.clamp(min=1)[:, None]
    hot = torch.zeros((T, 8), dtype=torch.float64).scatter_add_(1, idx.long(), torch.ones((T, 2), dtype=torch.float64))
    c = torch.zeros((S, 8), dtype=torch.float64).index_add_(0, seq, hot)
    assert torch.equal(rows.cpu().long(), n) and torch.equal(counts.cpu().double(), c)
    assert (probs.cpu().double() - want).abs().max() < 200 * U
    assert abs(float(loss[0]) - float((8 * c / (2 * n.clamp(min=1)[:, None]) * want).sum() / S)) < 400 * U
    dl = dlm.balance_backward(l.cuda(), counts, rows, 2, alpha=1.0, offsets=off.cuda())
    u = (8 / (2 * S * n.clamp(min=1).double() ** 2)[:, None] * c)[seq]
    g = p * (u - (u * p).sum(1, keepdim=True))
    assert ((dl.cpu().double() - g).abs() <= 300 * U * u.abs().amax(1, keepdim=True) + 2.0 ** -120).all()
    with pytest.raises(dlm.DLMError):
        dlm.balance(l.cuda(), idx.cuda(), offsets=torch.zeros(S + 2, dtype=torch.int32, device="cuda"))


def test_no_rows():
    for off in (None, torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda")):
        S = 1 if off is None else 2
        loss, counts, rows, probs = dlm.balance(torch.empty((0, 5), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                                                zeta=1.0, offsets=off, loss=torch.ones(2, device="cuda"),
                                                rows=torch.ones(S, dtype=torch.int32, device="cuda"))
        assert loss.tolist() == [0.0, 0.0] and not counts.any() and not rows.any() and not probs.any()
        assert dlm.balance_backward(torch.empty((0, 5), device="cuda"), counts, rows, 2, offsets=off).shape == (0, 5)


def test_balanced_router_has_alpha():
    """Equal scores and equal counts: the balance term is alpha, and nothing pulls."""
    E, T = 8, 64
    idx = torch.stack([torch.arange(T) % E, (torch.arange(T) + 3) % E], 1).int()
    loss, _, _, _, dl = _check(torch.zeros((T, E)), idx, "softmax", 0.25, 0.0, None)
    assert abs(float(loss[0]) - 0.25) < 1e-6 and float(dl.abs().max()) < 1e-9


def test_joint_batches():
    """Two halves with their counts and rows summed: gradients as from the whole batch."""
    l, idx = _inputs(200, 16, 2, torch.float32, 8)
    _, counts, rows, _, dl = _check(l, idx, "softmax", 0.1, 0.01, None)
    cs, rs = zip(*[dlm.balance(h.cuda(), i.cuda(), alpha=0.1, zeta=0.01)[1:3] for h, i in ((l[:77], idx[:77]), (l[77:], idx[77:]))])
    c, r = cs[0] + cs[1], rs[0] + rs[1]
    assert torch.equal(c, counts) and torch.equal(r, rows)
    got = torch.cat([dlm.balance_backward(h.cuda(), c, r, 2, alpha=0.1, zeta=0.01) for h in (l[:77], l[77:])])
    assert torch.equal(got, dl)


def test_same_bits_twice_in_a_dirty_workspace_and_on_another_stream():
    l, idx = _inputs(5000, 100, 6, torch.bfloat16, 2)
    off = torch.tensor([0, 17, 1000, 1001, 4990], dtype=torch.int32, device="cuda")
    x, i = l.cuda(), idx.cuda()
    want = dlm.balance(x, i, alpha=0.1, zeta=0.1, offsets=off)
    s = torch.cuda.Stream()
    for fill in (0x00, 0x5A, 0xFF):
        ws = torch.full((dlm.balance_workspace_size(5000, 100, 4),), fill, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        got = dlm.balance(x, i, alpha=0.1, zeta=0.1, offsets=off, workspace=ws, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_replayed_from_a_graph():
    """Route, loss and both gradients captured once: replays on new logits, with eager work between, equal eager calls."""
    l, _ = _inputs(3000, 64, 4, torch.float32, 4)
    x = l.cuda()
    off = torch.tensor([0, 1000, 2500], dtype=torch.int32, device="cuda")
    dg = torch.randn((3000, 4), generator=torch.Generator().manual_seed(1)).cuda()
    idx, g = dlm.route(x, 4)
    loss, counts, rows, probs = dlm.balance(x, idx, alpha=0.1, offsets=off)
    ws = torch.empty(dlm.balance_workspace_size(3000, 64, 2), dtype=torch.uint8, device="cuda")
    dl = torch.zeros_like(x)

    def step():
        dlm.route(x, 4, idx=idx, g=g)
        dlm.balance(x, idx, alpha=0.1, offsets=off, loss=loss, counts=counts, rows=rows, probs=probs, workspace=ws)
        dlm.route_backward(x, idx, dg, dlogits=dl)
        dlm.balance_backward(x, counts, rows, 4, alpha=0.1, offsets=off, dlogits=dl, accumulate=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(3):
        x.copy_(_inputs(3000, 64, 4, torch.float32, 40 + r)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (idx, loss, counts, rows, probs, dl)]
        for t in (loss, counts, rows, probs, dl):
            t.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (idx, loss, counts, rows, probs, dl)))


def test_past_2_32_logits():
    E = 512
    T = (1 << 32) // E + 100
    x = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    tail, ti = _inputs(150, E, 4, torch.bfloat16, 0)
    x[-150:] = tail.cuda()
    idx = torch.full((T, 4), -1, dtype=torch.int32, device="cuda")
    idx[-150:] = ti.cuda()
    off = torch.tensor([0, T - 150, T], dtype=torch.int32, device="cuda")
    print("balance", T, E, flush=True)
    loss, counts, rows, probs = dlm.balance(x, idx, alpha=0.1, zeta=0.1, offsets=off)
    one = dlm.balance(tail.cuda(), ti.cuda(), alpha=0.1, zeta=0.1)
    assert torch.equal(counts[1], one[1][0]) and rows.tolist() == [T - 150, 150]
    assert not counts[0].any() and (probs[0] - 1 / E).abs().max() < 9 * U / E
    dl = dlm.balance_backward(x, counts, rows, 4, alpha=0.1, zeta=0.1, offsets=off)
    ds = dlm.balance_backward(tail.cuda(), counts[1:].contiguous(), rows[1:].contiguous(), 4, alpha=0.05, zeta=0.05)
    assert torch.equal(dl[-150:], ds)
    assert (dl[:1000, :8].float() - 2 * 0.05 * math.log(E) / (T - 150) / E).abs().max() < 2.0 ** -8 * 2 * 0.05 * math.log(E) / (T - 150) / E


def _repeated(T, E, k, dtype, score, offsets):
    """T rows that are all one: (probs, loss) against that row's own scores, to their error and one rounding
    of the mean.  A sum's rounding then falls the same way every time, so one that is kept in fp32 over the
    batch is off by a share of its length: a hundred of 2^-24 after 500 rows."""
    row, _ = _inputs(1, E, 1, dtype, T % 1000 + E)
    p, _, lse, _, _ = ref.scores(row.double(), score)
    tol = (ref.relative(row.double(), p, score) + 2 * U) * p
    idx = torch.full((T, k), E // 3, dtype=torch.int32, device="cuda")
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    b = ref.borders(T, offsets)
    loss, counts, rows, probs = dlm.balance(row.cuda().expand(T, E).contiguous(), idx, score=score, offsets=off)
    lens = torch.tensor(b).diff()
    assert torch.equal(rows.cpu().long(), lens) and torch.equal(counts[:, E // 3].cpu().long(), lens * k)
    err = (probs.cpu().double() - p).abs()
    assert (err <= tol)[lens > 0].all(), float((err / (U * p))[lens > 0].max())
    # every slot of every row names one expert: f is E for it
    share = int((lens > 0).sum()) / (len(b) - 1)
    assert abs(float(loss[0]) - share * E * float(p[0, E // 3])) <= share * E * float(tol[0, E // 3] + 2 * U * p[0, E // 3])


@pytest.mark.parametrize("T,E,dtype,score,offsets", [
    (1 << 21, 512, torch.float32, "softmax", None), (1 << 21, 300, torch.bfloat16, "sigmoid", None),
    (1 << 21, 512, torch.bfloat16, "softmax", [0, 1 << 20, 1 << 20, (1 << 20) + 5, 1 << 21]),
    (1 << 24, 8, torch.float32, "sigmoid", [100, 1 << 23, 1 << 24])])
def test_long_batches_of_equal_rows(T, E, dtype, score, offsets):
    """Thousands of rows a lane, whose probabilities are no powers of two."""
    print("balance", T, E, flush=True)
    _repeated(T, E, 2, dtype, score, offsets)


def test_refusals_of_the_binding():
    x, idx = torch.zeros((4, 8), device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    _, counts, rows, _ = dlm.balance(x, idx)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for call in (lambda: dlm.balance(x.cpu(), idx), lambda: dlm.balance(x.t(), idx), lambda: dlm.balance(x, idx.long()),
                 lambda: dlm.balance(x, idx[:3]), lambda: dlm.balance(x, idx, offsets=off.long()),
                 lambda: dlm.balance(x, idx, offsets=off[:1]), lambda: dlm.balance(x, idx, counts=counts, offsets=off),
                 lambda: dlm.balance(x, idx, score="tanh"), lambda: dlm.balance(x, idx, loss=torch.zeros(1, device="cuda")),
                 lambda: dlm.balance_backward(x, counts, rows, 2, offsets=off),
                 lambda: dlm.balance_backward(x, counts, rows, 2, accumulate=True),
                 lambda: dlm.balance_backward(x, counts.float(), rows, 2),
                 lambda: dlm.balance_backward(x, counts, rows, 2, dlogits=torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")),
                 lambda: dlm.balance_backward(x, counts, rows, 2, dloss=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        dlm.balance(x.half(), idx)
    for call in (lambda: dlm.balance(x, idx, score="sigmoid", zeta=0.1), lambda: dlm.balance(x, idx, alpha=float("nan")),
                 lambda: dlm.balance(x, idx, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")),
                 lambda: dlm.balance_backward(x, counts, rows, 0), lambda: dlm.balance_backward(x, counts, rows, 2, dlogits=x)):
        with pytest.raises(dlm.DLMError):
            call()
