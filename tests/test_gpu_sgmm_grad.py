"""The SGMM's gradients on the GPU against the plain binary64 form.

Tolerances, with S the formula's sum over magnitudes and gamma_n the bound of an
n-term fp32 sum (gpu_util): u and w are sums of d_in and d_out products, the
coefficients s g u and s g w two more roundings, and in bf16 two bf16 terms
(hi to 2^-8 of the value, lo to 2^-8 of the rest: 2^-16); the last sum runs over
the rank (dx), the expert's slots twice (dA, dB: hi and lo) or rank and problems (dg):
  dA  (gamma(d_out + 2 slots + 8) + 2^-16) S       dB the same with d_in
  dx  (gamma(d_out + 4 r + 8) + 2^-16) S, and bf16's rounding 2^-8 of the result
  dg  gamma(d_in + d_out + 2 r + problems + 8) S
fp32 has no 2^-16 and no 2^-8 but fp32's own rounding.  The bounds above are the
worst case; over random signs the split's error adds up like the values do, so
the norms of dA and dB are also held to 2^-14 of the result's (fp32: 2^-18)."""
import numpy as np
import pytest
import torch

import dynamic_lora_moe_amd as dlm
import grad_ref as ref
from gpu_util import gamma

pytestmark = pytest.mark.gpu
SPLIT = 2.0 ** -16


def _rnd(shape, dtype, std, gen):
    return (torch.randn(shape, generator=gen) * std).to(dtype)


def _sets(T, E, gen, empty=0.1, both=0.05, dup=0.0):
    idx = torch.randint(0, E, (T, 2), generator=gen, dtype=torch.int32)
    if E > 1:
        same = (idx[:, 0] == idx[:, 1]) & (torch.rand(T, generator=gen) >= dup)
        idx[same, 1] = (idx[same, 0] + 1) % E
    idx[torch.rand(T, generator=gen) < empty, 1] = -1
    idx[torch.rand(T, generator=gen) < empty, 0] = -1
    idx[torch.rand(T, generator=gen) < both] = -1
    return idx, torch.rand((T, 2), generator=gen) - 0.25


class Case:
    """A group of problems with their gradients' buffers, device and host."""

    def __init__(self, T, shapes, E, r, dtype, seed=0, scale=1.5, rows=None, **sets):
        gen = torch.Generator().manual_seed(seed)
        self.T, self.E, self.r, self.dtype, self.scale = T, E, r, dtype, scale
        n = T if rows is None else rows
        self.idx, self.g = _sets(T, E, gen, **sets)
        self.x = [_rnd((n, i), dtype, 1.0, gen) for o, i in shapes]
        self.A = [_rnd((E, r, i), dtype, i ** -0.5, gen) for o, i in shapes]
        self.B = [_rnd((E, o, r), dtype, 0.3, gen) for o, i in shapes]
        self.dy = [_rnd((n, o), dtype, 1.0, gen) for o, i in shapes]
        self.dx0 = [_rnd((n, i), dtype, 1.0, gen) for o, i in shapes]
        self.shapes = shapes

    def bind(self, dx=None):
        up = lambda ts: [t.cuda() for t in ts]  # noqa: E731
        self.dev = list(zip(up(self.x), up(self.A), up(self.B), [torch.zeros_like(t).cuda() for t in self.dy]))
        self.ddy, self.ddx = up(self.dy), up(self.dx0) if dx is None else dx
        self.dA = [torch.full(t.shape, 9.0, device="cuda") for t in self.A]
        self.dB = [torch.full(t.shape, 9.0, device="cuda") for t in self.B]
        self.dg = torch.full((self.T, 2), 9.0, device="cuda")
        self.grp = dlm.SgmmGroup(self.dev, self.E, self.r, self.scale)
        self.grp.bind_grads(self.ddy, self.ddx, self.dA, self.dB)
        return self

    def run(self, **kw):
        ws = self.grp.backward(self.idx.cuda(), self.g.cuda(), self.dg, **kw)
        torch.cuda.synchronize()
        return ws

    def refs(self):
        T = self.T
        return [ref.backward(x[:T], self.idx, self.g, A, B, dy[:T], self.scale)
                for x, A, B, dy in zip(self.x, self.A, self.B, self.dy)]

    def check(self, base=0.0):
        bf = self.dtype == torch.bfloat16
        split, u = (SPLIT, 2.0 ** -8) if bf else (0.0, 2.0 ** -24)
        slots = max([int((self.idx == e).sum()) for e in range(self.E)])
        dg = torch.zeros((self.T, 2), dtype=torch.float64)
        dgm = torch.zeros_like(dg)
        terms = 0
        for p, ((o, i), (out, mag)) in enumerate(zip(self.shapes, self.refs())):
            for name, got, want, m, n in (("dA", self.dA[p], out[1], mag[1], o), ("dB", self.dB[p], out[2], mag[2], i)):
                got = got.cpu().double()
                err = (got - base - want).abs()
                tol = (gamma(n + 2 * slots + 8) + split) * m + 2.0 ** -23 * abs(base)
                assert (err <= tol).all(), (name, p, float((err - tol).max()))
                if base == 0.0 and want.norm() > 0 and want.numel() >= 256:
                    assert err.norm() <= (2.0 ** -14 if bf else 2.0 ** -18) * want.norm(), (name, p)
            if self.ddx[p] is not None:
                want = self.dx0[p][:self.T].double() + out[0]
                err = (self.ddx[p][:self.T].cpu().double() - want).abs()
                tol = (gamma(o + 4 * self.r + 8) + split) * (mag[0] + self.dx0[p][:self.T].double().abs() * (1 - bf)) + u * want.abs()
                assert (err <= tol + u * tol).all(), ("dx", p, float((err - tol).max()))
                assert torch.equal(self.ddx[p][self.T:].cpu(), self.dx0[p][self.T:])
                none = (self.idx < 0).all(1)
                assert torch.equal(self.ddx[p][:self.T].cpu()[none], self.dx0[p][:self.T][none])
            dg += out[3]
            dgm += mag[3]
            terms = max(terms, o + i)
        err = (self.dg.cpu().double() - dg).abs()
        assert (err <= gamma(terms + 2 * self.r + len(self.shapes) + 8) * dgm).all(), ("dg", float(err.max()))
        assert (self.dg.cpu()[self.idx < 0] == 0).all()


BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 31, 32, 33, 63, 64, 65, 200, 1000, 2500])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_length(T, dtype):
    print(T, dtype, flush=True)
    c = Case(T, [(136, 264)], 8, 16, dtype, seed=T).bind()
    c.run()
    c.check()


@pytest.mark.parametrize("r", [1, 2, 3, 4, 7, 8, 12, 16, 17, 24, 31, 32, 40, 48, 63, 64, 65, 80, 96, 127, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_rank(r, dtype):
    print(r, dtype, flush=True)
    c = Case(70, [(72, 200)], 4, r, dtype, seed=r).bind()
    c.run()
    c.check()


@pytest.mark.parametrize("E", [1, 2, 3, 16, 31, 32])
@pytest.mark.parametrize("dup", [0.0, 1.0])
def test_every_bank_size(E, dup):
    """Up to 32 experts, with rows that name one expert twice."""
    print(E, dup, flush=True)
    c = Case(300, [(64, 128)], E, 16, BF, seed=E, dup=dup).bind()
    c.run()
    c.check()


@pytest.mark.parametrize("o,i", [(8, 8), (8, 4096), (4104, 8), (2056, 1032), (128, 6152), (6152, 136), (1000, 120)])
@pytest.mark.parametrize("r", [16, 64, 96])
def test_shapes_bf16(o, i, r):
    """One to four K slices on either side, widths that end inside a column block."""
    print(o, i, r, flush=True)
    c = Case(130, [(o, i)], 6, r, BF, seed=o + i).bind()
    c.run()
    c.check()


@pytest.mark.parametrize("o,i", [(1, 1), (3, 5), (129, 257), (1000, 77)])
def test_shapes_f32(o, i):
    print(o, i, flush=True)
    c = Case(41, [(o, i)], 3, 5, F32, seed=o + i).bind()
    c.run()
    c.check()


@pytest.mark.parametrize("dtype,r", [(BF, 16), (BF, 96), (F32, 6)])
def test_groups(dtype, r):
    """Seven projections of a layer's shapes (scaled down), one segmentation, dg over all of them."""
    shapes = [(256, 256)] * 4 + [(688, 256)] * 2 + [(256, 688)]
    c = Case(150, shapes, 8, r, dtype, seed=3).bind()
    c.run()
    c.check()


def test_many_rows():
    """Past the segmentation's one-launch limit, one expert chosen by most rows."""
    print("rows 9000", flush=True)
    c = Case(9000, [(64, 72)], 8, 8, BF, seed=4)
    c.idx[:7000, 0] = 5
    c.idx[:7000, 1] = torch.where(c.idx[:7000, 1] == 5, 6, c.idx[:7000, 1].long()).int()
    c.bind()
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_without_experts(dtype):
    """No row has a set: zero bank gradients, dx untouched, dg zero."""
    c = Case(40, [(64, 64)], 4, 8, dtype)
    c.idx[:] = -1
    c.bind()
    c.run()
    c.check()
    assert (c.dA[0] == 0).all() and (c.dB[0] == 0).all() and (c.dg == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_empty_rows_hold_does_not_matter(dtype):
    """Infinities and NaN in rows without a set, and in rows behind T, reach nothing."""
    c = Case(50, [(136, 128)], 4, 16, dtype, rows=64).bind()
    none = (c.idx < 0).all(1)
    assert none.any()
    for t, d in ((c.x[0], c.dev[0][0]), (c.dy[0], c.ddy[0])):
        t[:50][none] = float("nan")
        t[50:] = float("inf")
        d.copy_(t)
        t[:50][none] = 0  # the plain form leaves these rows out by index, not by value
    c.run(T=50)
    c.check()


def test_infinities_stay_with_their_expert():
    """One row's infinite dy: only its experts' gradients and its own dx lose their values."""
    c = Case(100, [(64, 64)], 8, 16, BF, empty=0.0, both=0.0).bind()
    e = set(c.idx[17].tolist())
    c.ddy[0][17, 3] = float("inf")
    c.run()
    for k in range(8):
        assert torch.isfinite(c.dA[0][k]).all() == (k not in e)
        assert torch.isfinite(c.dB[0][k]).all() == (k not in e)
    fin = torch.isfinite(c.ddx[0]).all(1).cpu()
    assert not fin[17] and fin[torch.arange(100) != 17].all()


@pytest.mark.parametrize("T,E,r,dup", [(1, 2, 64, 0.0), (5, 32, 40, 1.0), (129, 2, 64, 0.5), (700, 2, 48, 0.0),
                                       (700, 32, 64, 1.0), (1300, 6, 128, 0.2), (1300, 16, 33, 0.0), (9000, 3, 64, 0.0)])
def test_ranks_above_32(T, E, r, dup):
    """Sums over the experts' slot lists: groups of slots that end inside one, a single slot, one expert twice in a row."""
    print(T, E, r, flush=True)
    c = Case(T, [(200, 136), (72, 2056)] if T < 2000 else [(72, 136)], E, r, BF, seed=T + r, dup=dup).bind()
    c.run()
    c.check()


def test_rows_without_experts_at_rank_64():
    c = Case(40, [(64, 72)], 4, 64, BF)
    c.idx[:] = -1
    c.bind()
    c.run()
    c.check()
    assert (c.dA[0] == 0).all() and (c.dB[0] == 0).all() and (c.dg == 0).all()


@pytest.mark.parametrize("i", [64, 72])
def test_infinities_stay_with_their_row_and_rank(i):
    """Rank 64, widths that end inside a step: one row's infinite x, and one infinity at the end of a bank's row."""
    c = Case(100, [(i, i)], 8, 64, BF, empty=0.0, both=0.0).bind()
    e = set(c.idx[17].tolist())
    c.dev[0][0][17, i - 1] = float("inf")
    c.run()
    fin = torch.isfinite(c.dg).all(1).cpu()
    assert not fin[17] and fin[torch.arange(100) != 17].all()
    for k in range(8):
        assert torch.isfinite(c.dA[0][k]).all() == (k not in e)
        assert torch.isfinite(c.dB[0][k]).all() == (k not in e)
    c = Case(100, [(i, i)], 8, 64, BF, empty=0.0, both=0.0).bind()
    c.dev[0][1][3, 5, i - 1] = float("inf")  # A of expert 3, rank 5: only that rank's u, so only dB[3][:, 5]
    c.run()
    assert torch.isfinite(c.dA[0]).all()
    want = torch.ones((8, 64), dtype=torch.bool)
    want[3, 5] = False
    assert torch.equal(torch.isfinite(c.dB[0]).all(1).cpu(), want)


@pytest.mark.parametrize("r", [4, 16, 24, 64, 100])
def test_coefficients_keep_every_bit_of_fp32(r):
    """One row an expert, x and dy a single power of two, the banks powers of two: u and w are exact, and
    s g w and s g u are gates of 24 significant bits.  Three bf16 terms hold those whole and add up without a
    rounding, so dA and dB are exact (two terms would be 2^-17 of an element off in most of them)."""
    E = T = 32
    d = 72
    gen = torch.Generator().manual_seed(r)
    row = torch.arange(T)

    def pow2(*s):
        return torch.exp2(torch.randint(-2, 3, s, generator=gen).float()) * (2 * torch.randint(0, 2, s, generator=gen) - 1)

    x, dy = torch.zeros(T, d), torch.zeros(T, d)
    x[row, torch.randint(0, d, (T,), generator=gen)] = pow2(T)
    dy[row, torch.randint(0, d, (T,), generator=gen)] = pow2(T)
    A, B = pow2(E, r, d), pow2(E, d, r)
    idx = torch.stack([torch.randperm(E, generator=gen), torch.full((T,), -1)], 1).int()
    g = torch.rand((T, 2), generator=gen) / 2 + 0.5
    up = lambda t: t.bfloat16().cuda()  # noqa: E731
    dA, dB = torch.empty((E, r, d), device="cuda"), torch.empty((E, d, r), device="cuda")
    grp = dlm.SgmmGroup([(up(x), up(A), up(B), up(torch.zeros(T, d)))], E, r, 1.0)
    grp.bind_grads([up(dy)], None, [dA], [dB])
    grp.backward(idx.cuda(), g.cuda())
    torch.cuda.synchronize()
    _, wA, wB, _ = ref.backward(x, idx, g, A, B, dy, 1.0)[0]
    assert torch.equal(dA.cpu().double(), wA) and torch.equal(dB.cpu().double(), wB)


@pytest.mark.parametrize("T,r", [(300, 16), (300, 64), (600, 16)])
def test_bank_gradients_are_nearer_than_two_terms_would_be(T, r):
    """The norms of dA and dB against the plain form's, u and w being sums of eight products.  An element is
    the sum of n = T / 4 slots: with 7 roundings of u or w, 2 of the coefficient and n of the sum, each 2^-24 /
    sqrt(3) in the root mean square, fp32 leaves sqrt(n + 9) times that, at most 2^-21.1 of the norm.  A two-term
    form worked out here leaves more than the 2^-20 that is allowed."""
    c = Case(T, [(8, 8)], 8, r, BF, seed=T + r, empty=0.0, both=0.0).bind()
    c.run()
    out, _ = c.refs()[0]
    x, A, B, dy = (t[0].double() for t in (c.x, c.A, c.B, c.dy))
    two = [torch.zeros_like(A), torch.zeros_like(B)]
    for t in range(T):
        for k in (0, 1):
            e, s = int(c.idx[t, k]), c.scale * float(c.g[t, k])
            for grad, co, row in ((two[0], s * (dy[t] @ B[e]), x[t]), (two[1], s * (A[e] @ x[t]), dy[t])):
                hi = co.bfloat16().double()
                co = hi + (co - hi).bfloat16().double()
                grad[e] += torch.outer(co, row) if grad is two[0] else torch.outer(row, co)
    for got, want, short in ((c.dA[0], out[1], two[0]), (c.dB[0], out[2], two[1])):
        assert (got.cpu().double() - want).norm() <= 2.0 ** -20 * want.norm()
        assert (short - want).norm() > 2.0 ** -20 * want.norm()


@pytest.mark.parametrize("dtype,E,r,T,shape", [(BF, 8, 16, 100, (64, 64)), (BF, 8, 64, 100, (72, 200)), (BF, 8, 128, 100, (64, 72)),
                                               (BF, 32, 16, 300, (64, 136)), (BF, 32, 64, 300, (64, 64)), (BF, 32, 5, 300, (64, 2056)),
                                               (BF, 12, 100, 200, (64, 72)), (F32, 8, 6, 100, (40, 33))])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_bank_that_is_not_finite_stays_with_its_rows(dtype, E, r, T, shape, value):
    """One element of one expert's A (every matrix tile of its rows holds others' too): dx of the rows that
    choose it is lost in that column, everything else is as if that expert's terms were elsewhere."""
    o, i = shape
    col, rank = i - 3, r - 1
    c = Case(T, [shape], E, r, dtype, empty=0.1, both=0.0).bind()
    c.dev[0][1][3, rank, col] = value
    c.run()
    mine = (c.idx == 3).any(1) & (c.g[torch.arange(T)[:, None], torch.arange(2)] != 0).any(1)
    assert mine.any() and (~mine).any()
    got = c.ddx[0].cpu()
    assert not torch.isfinite(got[mine, col]).any()
    # what the value cannot reach, against the plain form of the banks as they were
    out, mag = c.refs()[0]
    want = c.dx0[0].double() + out[0]
    bf = dtype == BF
    u = 2.0 ** -8 if bf else 2.0 ** -24
    tol = (gamma(o + 4 * r + 8) + (SPLIT if bf else 0.0)) * (mag[0] + c.dx0[0].double().abs() * (1 - bf)) + u * want.abs()
    free = torch.ones_like(got, dtype=torch.bool)
    free[mine, col] = False
    err = (got.double() - want).abs()
    assert (err[free] <= (tol + u * tol)[free]).all()
    other = (c.idx != 3).all(1)
    dg, dgm = out[3], mag[3]
    assert ((c.dg.cpu().double() - dg).abs()[other] <= gamma(o + i + 2 * r + 9) * dgm[other]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_accumulate(dtype):
    c = Case(90, [(72, 136), (64, 64)], 5, 12, dtype).bind()
    for t in c.dA + c.dB:
        t.fill_(2.0)
    c.run(accumulate=True)
    c.check(base=2.0)


def test_shared_dx_and_unwanted_dx():
    """q, k, v of one x: the shares of one dx add up, each rounded once; a None entry is left out."""
    gen = torch.Generator().manual_seed(1)
    c = Case(80, [(64, 128), (32, 128), (64, 128), (128, 64)], 4, 16, BF)
    c.x[1] = c.x[2] = c.x[0]
    dx = _rnd((80, 128), BF, 1.0, gen)
    dev = dx.cuda()
    c.bind(dx=[dev, dev, dev, None])
    c.run()
    refs = c.refs()
    want, tol = dx.double(), 0.0
    for (o, i), (out, mag) in list(zip(c.shapes, refs))[:3]:
        want = want + out[0]
        tol = tol + (gamma(o + 4 * 16 + 8) + SPLIT) * mag[0] + 2.0 ** -8 * want.abs()
    assert ((dev.cpu().double() - want).abs() <= tol * (1 + 3 * 2.0 ** -8)).all()
    c.ddx = [None] * 4
    c.check()


def test_rows_behind_the_last_sequence():
    """T smaller than the buffers: rows from T on are read and written nowhere."""
    c = Case(33, [(64, 72)], 4, 16, BF, rows=70).bind()
    c.run(T=33)
    c.check()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", ["index", "negative", "gate"])
def test_rejected_sets_change_nothing(dtype, bad):
    c = Case(60, [(64, 64)], 4, 8, dtype, empty=0.0, both=0.0).bind()
    good_idx, good_g = c.idx.clone(), c.g.clone()
    if bad == "index":
        c.idx[7, 1] = 4
    elif bad == "negative":
        c.idx[7, 0] = -2
    else:
        c.g[7, 0] = float("nan")
    ws = c.run()
    assert dlm.sgmm_status(ws) == dlm.DLM_EDEVICE
    assert (c.dA[0] == 9).all() and (c.dB[0] == 9).all() and (c.dg == 9).all()
    assert torch.equal(c.ddx[0].cpu(), c.dx0[0])
    c.idx, c.g = good_idx, good_g
    ws = c.run()
    assert dlm.sgmm_status(ws) == dlm.DLM_OK
    c.check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_workspace_serves_fewer_rows(dtype):
    """A workspace for the largest batch, used for smaller ones (which cut K and the lists otherwise)."""
    c = Case(3000, [(2056, 264)], 8, 16, dtype).bind()
    ws = c.grp.backward_workspace(3000)
    full = c.idx.clone()
    for T in (3000, 1024, 300, 64, 7, 1):
        assert c.grp.backward_workspace(T).numel() <= ws.numel()
        for t, d in zip(c.ddx, c.dx0):
            t.copy_(d)
        ws.fill_(0x7F)
        c.T, c.idx = T, full[:T]
        gate = c.g
        c.g = gate[:T]
        c.dg = torch.empty((T, 2), device="cuda")
        c.run(workspace=ws)
        c.check()
        c.g = gate


@pytest.mark.parametrize("r", [16, 64, 128])
def test_a_workspace_serves_every_smaller_batch(r):
    c = Case(8, [(2056, 264), (64, 8200)], 8, r, BF).bind()
    sizes = [c.grp.backward_workspace(T).numel() for T in (*range(1, 600), *range(600, 20000, 97))]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("r", [16, 64])
def test_no_dx_at_all(r):
    """Nothing asks for dx: the coefficients are a launch of their own."""
    c = Case(300, [(72, 136), (64, 64)], 6, r, BF).bind(dx=[None, None])
    c.run()
    c.check()


@pytest.mark.parametrize("r", [16, 64])
def test_tied_banks_and_shared_dx(r):
    """Two problems of one A, B and x with one dx: every gradient buffer has its own problem's share."""
    c = Case(200, [(64, 128), (64, 128)], 4, r, BF)
    c.x[1], c.A[1], c.B[1] = c.x[0], c.A[0], c.B[0]
    c.bind()
    x, A, B, _ = c.dev[0]
    c.dev = [(x, A, B, c.dev[0][3]), (x, A, B, c.dev[1][3])]
    dx = c.dx0[0].cuda()
    c.grp = dlm.SgmmGroup(c.dev, c.E, r, c.scale)
    c.grp.bind_grads(c.ddy, [dx, dx], c.dA, c.dB)
    c.run()
    want, tol = c.dx0[0].double(), 0.0
    for (o, i), (out, mag) in zip(c.shapes, c.refs()):
        want = want + out[0]
        tol = tol + (gamma(o + 4 * r + 8) + SPLIT) * mag[0] + 2.0 ** -8 * want.abs()
    assert ((dx.cpu().double() - want).abs() <= tol * (1 + 3 * 2.0 ** -8)).all()
    c.ddx = [None, None]
    c.check()


def test_a_rejected_set_changes_nothing_at_rank_64():
    c = Case(300, [(64, 72)], 4, 64, BF, empty=0.0, both=0.0).bind()
    c.idx[7, 1] = 4
    before = [t.clone() for t in c.ddx + c.dA + c.dB + [c.dg]]
    ws = c.run()
    assert dlm.sgmm_status(ws) == dlm.DLM_EDEVICE
    assert all(torch.equal(x, y) for x, y in zip(before, c.ddx + c.dA + c.dB + [c.dg]))


def test_no_rows():
    c = Case(16, [(64, 64)], 4, 8, BF).bind()
    e = torch.empty((0, 2), device="cuda")
    c.grp.backward(e.int(), e, accumulate=True)
    torch.cuda.synchronize()
    assert (c.dA[0] == 9).all()
    c.grp.backward(e.int(), e)
    torch.cuda.synchronize()
    assert (c.dA[0] == 0).all() and (c.dB[0] == 0).all() and torch.equal(c.ddx[0].cpu(), c.dx0[0])


@pytest.mark.parametrize("dtype,r", [(BF, 16), (F32, 16), (BF, 64), (BF, 128)])
def test_same_bits_every_time_on_any_stream_and_replayed(dtype, r):
    """Eager, on another stream, and replayed from a graph with eager work between the replays."""
    c = Case(500, [(256, 136), (72, 2056)], 8, r, dtype).bind()
    idx, g = c.idx.cuda(), c.g.cuda()
    ws = c.grp.backward_workspace(c.T)
    outs = c.ddx + c.dA + c.dB + [c.dg]
    c.grp.backward(idx, g, c.dg, workspace=ws)
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]

    def reset():
        for t, d in zip(c.ddx, c.dx0):
            t.copy_(d)
        for t in c.dA + c.dB + [c.dg]:
            t.fill_(float("nan"))
        ws.fill_(0x5A)
        torch.cuda.synchronize()

    reset()
    s = torch.cuda.Stream()
    c.grp.backward(idx, g, c.dg, workspace=ws, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.grp.backward(idx, g, c.dg, workspace=ws)
    for _ in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_two_groups_at_once():
    """Two handles with workspaces of their own, on two streams without an order between them."""
    cs = [Case(900, [(264, 136), (72, 2056)], 8, r, BF, seed=r).bind() for r in (16, 64)]
    args = [(c.idx.cuda(), c.g.cuda(), c.grp.backward_workspace(c.T)) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for (idx, g, ws), c, s in zip(args, cs, streams):
        c.grp.backward(idx, g, c.dg, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for c in cs:
        c.check()


def test_reads_the_banks_as_they_are():
    """Banks changed in place between calls (as an optimiser does): no repack is needed for the gradients."""
    c = Case(70, [(64, 72)], 4, 16, BF).bind()
    c.run()
    for t, (x, A, B, y) in zip(range(1), c.dev):
        A.mul_(-2.0)
        B.add_(0.5)
        c.A[0], c.B[0] = A.cpu(), B.cpu()
    for t, d in zip(c.ddx, c.dx0):
        t.copy_(d)
    c.run()
    c.check()


def test_gradients_against_differences():
    """Directional differences of the product in binary64 against the kernels' fp32 gradients: the
    product is linear in x, g, A and B each, so a central difference has no truncation error, and
    what is left is the gradients' own bound."""
    c = Case(12, [(24, 40)], 3, 4, F32, seed=2).bind()
    for t in c.ddx:
        t.zero_()
    c.run()
    gen = torch.Generator().manual_seed(0)
    x, A, B, g, dy = c.x[0].double(), c.A[0].double(), c.B[0].double(), c.g.double(), c.dy[0].double()
    for which, grad in (("x", c.ddx[0]), ("A", c.dA[0]), ("B", c.dB[0]), ("g", c.dg)):
        v = torch.randn(grad.shape, generator=gen).double()
        f = lambda s: (ref.forward(x + s * v if which == "x" else x, c.idx, g + s * v if which == "g" else g,  # noqa: E731
                                   A + s * v if which == "A" else A, B + s * v if which == "B" else B, c.scale) * dy).sum()
        want = (f(0.5) - f(-0.5)).item()
        got = (grad.cpu().double() * v).sum().item()
        mag = (grad.cpu().double() * v).abs().sum().item()
        assert abs(got - want) <= 2.0 ** -16 * mag


def test_refusals_of_the_binding():
    c = Case(16, [(64, 64), (64, 64)], 4, 8, BF).bind()
    idx, g = c.idx.cuda(), c.g.cuda()
    fresh = dlm.SgmmGroup(c.dev, 4, 8, 1.0)
    with pytest.raises(dlm.DLMError):
        fresh.backward(idx, g, workspace=c.grp.backward_workspace(16))
    with pytest.raises(ValueError):
        fresh.bind_grads(c.ddy[:1], c.ddx, c.dA, c.dB)
    with pytest.raises(ValueError):
        fresh.bind_grads(c.ddy, c.ddx, [t.bfloat16() for t in c.dA], c.dB)
    with pytest.raises(ValueError):
        fresh.bind_grads([t[:8] for t in c.ddy], c.ddx, c.dA, c.dB)
    with pytest.raises(dlm.DLMError):
        c.grp.backward(idx, g, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        c.grp.backward(idx, g, T=17)
    with pytest.raises(ValueError):
        c.grp.backward(idx, g, torch.empty((15, 2), device="cuda"))
    # a written buffer that is also read, or written twice
    for bad in (dict(dys=c.ddy, dxs=[c.dev[0][0], None], dAs=c.dA, dBs=c.dB),
                dict(dys=c.ddy, dxs=[c.ddy[0], None], dAs=c.dA, dBs=c.dB),
                dict(dys=c.ddy, dxs=c.ddx, dAs=[c.dA[0], c.dA[0]], dBs=c.dB)):
        fresh.bind_grads(**bad)
        with pytest.raises(dlm.DLMError):
            fresh.backward(idx, g, workspace=c.grp.backward_workspace(16))
