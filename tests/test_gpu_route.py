"""Routing from logits and its gradient on the GPU against the plain binary64
forms: the choice exactly, the weights to half a unit of fp32, the gradient to
the rounding of its type.

Tolerances.  g: binary64 inside, one rounding to fp32, so 2^-24 of the value
plus what binary64 leaves (a few 2^-52 of scale).  dlogits: one rounding to its
type, eps / 2 of the value (fp32 2^-24, bf16 2^-8), plus binary64's remainder:
the gradient is a difference of terms up to |scale| * max|dg| * (k + 1) in size,
whose own relative errors are below 2^-44 (E + k operations of 2^-52 each)."""
import numpy as np
import pytest
import torch

import dynamic_lora_moe_amd as dlm
import route_ref as ref

pytestmark = pytest.mark.gpu

# a bound for the binary64 part of every comparison, relative to the largest term
R64 = 2.0 ** -44


def _logits(T, E, dtype, seed, masked=0.0, pitch=0):
    gen = torch.Generator().manual_seed(seed)
    l = torch.randn((T, E), generator=gen) * 1.5
    if masked:
        l[torch.rand((T, E), generator=gen) < masked] = -float("inf")
    l = l.to(dtype)
    if pitch:
        wide = torch.zeros((T, pitch), dtype=dtype, device="cuda")
        wide[:, :E] = l.cuda()
        return l, wide[:, :E]
    return l, l.cuda()


def _check(l, dev, k, bias=None, seed=0, **kw):
    T, E = l.shape
    counts = torch.full((E,), 7, dtype=torch.int32, device="cuda")
    idx, g = dlm.route(dev, k, bias=None if bias is None else bias.cuda(), counts=counts, **kw)
    torch.cuda.synchronize()
    ln = l.double().numpy()
    ri, rg = ref.route(ln, k, bias=None if bias is None else bias.double().numpy(), **kw)
    assert np.array_equal(idx.cpu().numpy(), ri)
    scale = abs(kw.get("scale", 1.0))
    err = np.abs(g.cpu().double().numpy() - rg)
    assert (err <= 2.0 ** -24 * np.abs(rg) + R64 * scale + 2.0 ** -149).all(), err.max()
    assert np.array_equal(counts.cpu().numpy(), 7 + np.bincount(ri[ri >= 0], minlength=E))
    back = {q: kw[q] for q in ("score", "renorm", "scale") if q in kw}
    dg = torch.randn((T, k), generator=torch.Generator().manual_seed(seed + 1))
    dl = dlm.route_backward(dev, idx, dg.cuda(), **back)
    rd = ref.route_backward(ln, ri, dg.double().numpy(), **back)
    half = torch.finfo(l.dtype).eps / 2
    err = np.abs(dl.cpu().double().numpy() - rd)
    assert (err <= half * np.abs(rd) + R64 * scale * 8 * (k + 1) + 2.0 ** -133).all(), err.max()
    return idx, g


@pytest.mark.parametrize("E", [1, 2, 7, 8, 9, 16, 24, 31, 32, 33, 60, 64, 100, 128, 129, 200, 256, 264, 384, 511, 512])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_width(E, score, renorm, dtype):
    l, dev = _logits(37, E, dtype, E)
    _check(l, dev, min(E, 6), score=score, renorm=renorm, scale=1.5)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(3)) * 0.3
    _check(l, dev, min(E, 3), bias=bias, score=score, renorm=renorm)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 257, 1000])
@pytest.mark.parametrize("E,k", [(8, 2), (60, 4), (256, 8), (512, 16), (16, 16)])
def test_every_length(T, E, k):
    l, dev = _logits(T, E, torch.float32, T + E)
    _check(l, dev, k)


@pytest.mark.parametrize("E,groups,keep,top", [(256, 8, 4, 2), (256, 8, 4, 1), (64, 32, 5, 2), (64, 32, 32, 1), (32, 32, 9, 1),
                                               (60, 4, 2, 2), (100, 10, 3, 2), (512, 2, 1, 2), (512, 32, 3, 1), (16, 16, 3, 2),
                                               (14, 2, 1, 1), (128, 32, 8, 2), (32, 16, 4, 2), (4, 2, 1, 2)])
@pytest.mark.parametrize("score,biased", [("sigmoid", True), ("softmax", False), ("sigmoid", False), ("softmax", True)])
def test_groups(E, groups, keep, top, score, biased):
    l, dev = _logits(70, E, torch.float32, E + groups)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(5)) * 0.2 if biased else None
    k = min(keep * (E // groups), 6)
    _check(l, dev, k, bias=bias, score=score, n_groups=groups, keep_groups=keep, group_top=top, scale=2.5)


@pytest.mark.parametrize("T,E,groups,keep", [(33000, 32, 1, 1), (33000, 32, 4, 2), (17000, 60, 1, 1), (17000, 64, 4, 2),
                                             (17000, 60, 10, 3), (8300, 128, 1, 1), (8300, 128, 4, 2), (8300, 100, 4, 1),
                                             (4200, 256, 1, 1), (4200, 256, 8, 4), (4200, 256, 32, 9)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_rows(T, E, groups, keep, dtype):
    """Enough rows that a lane holds 16 experts."""
    l, dev = _logits(T, E, dtype, T)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(5)) * 0.2
    for b, score, k in ((None, "softmax", 2), (bias, "sigmoid", 6)):
        _check(l, dev, k, bias=b, score=score, n_groups=groups, keep_groups=keep, group_top=2, renorm=k == 6)


@pytest.mark.parametrize("E,groups,keep,top", [(512, 4, 2, 2), (512, 32, 7, 2), (128, 8, 3, 1), (48, 3, 2, 2), (96, 2, 1, 2),
                                               (32, 2, 1, 1), (320, 20, 6, 2), (192, 3, 2, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [3, 8, 13])
def test_groups_of_whole_lanes(E, groups, keep, top, dtype, k):
    """Groups of 16 experts and more, whose lanes' lists rank them; the bias at an odd address."""
    l, dev = _logits(70, E, dtype, E + groups + k)
    l[3, : E // groups] = -float("inf")
    l[4] = -float("inf")
    dev.copy_(l)
    k = min(keep * (E // groups), k)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(k)) * 0.3
    for b in (None, bias):
        for score in ("softmax", "sigmoid"):
            _check(l, dev, k, bias=b, score=score, n_groups=groups, keep_groups=keep, group_top=top, scale=2.5)
    odd = torch.zeros(E + 1).cuda()
    odd[1:] = bias
    kw = dict(score="sigmoid", n_groups=groups, keep_groups=keep, group_top=top)
    i1, g1 = dlm.route(dev, k, bias=odd[1:], **kw)
    i2, g2 = dlm.route(dev, k, bias=bias.cuda(), **kw)
    assert torch.equal(i1, i2) and torch.equal(g1, g2)


@pytest.mark.parametrize("masked", [0.3, 0.9, 1.0])
@pytest.mark.parametrize("E,groups,keep", [(8, 1, 1), (60, 4, 2), (256, 8, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_rows_with_few_or_no_experts(masked, E, groups, keep, score):
    """Rows whose mask leaves fewer than k experts end in empty slots; rows it leaves empty have only those."""
    l, dev = _logits(65, E, torch.bfloat16, 11, masked=masked)
    for renorm in (True, False):
        idx, g = _check(l, dev, 4, score=score, n_groups=groups, keep_groups=keep, renorm=renorm)
        assert torch.isfinite(g).all() and (g[idx < 0] == 0).all()
        if masked == 1.0:
            assert (idx == -1).all()


@pytest.mark.parametrize("dtype,E,pitch", [(torch.float32, 8, 12), (torch.float32, 8, 9), (torch.bfloat16, 64, 72),
                                           (torch.bfloat16, 60, 61), (torch.float32, 256, 1000), (torch.bfloat16, 250, 256)])
def test_row_pitch(dtype, E, pitch):
    """Rows inside a wider matrix, aligned or not, in and out; what lies between the rows stays as it is."""
    l, dev = _logits(33, E, dtype, 2, pitch=pitch)
    idx, _ = _check(l, dev, 2)
    wide = torch.full((33, pitch), 5.0, dtype=dtype, device="cuda")
    dg = torch.randn((33, 2), generator=torch.Generator().manual_seed(0)).cuda()
    dlm.route_backward(dev, idx, dg, dlogits=wide[:, :E])
    assert torch.equal(wide[:, :E], dlm.route_backward(dev.contiguous(), idx, dg))
    assert (wide[:, E:] == 5.0).all()


def test_ties_go_to_the_lower_index():
    l = torch.zeros((5, 100))
    l[1, 50:] = 1.0
    l[2] = torch.tensor([float(i % 3) for i in range(100)])
    l[3, ::2] = -0.0  # equal to +0
    l[4] = -float("inf")
    idx, g = _check(l, l.cuda(), 4)
    assert idx[0].tolist() == [0, 1, 2, 3] and idx[1].tolist() == [50, 51, 52, 53] and idx[2].tolist() == [2, 5, 8, 11]
    assert idx[3].tolist() == [0, 1, 2, 3]
    _check(l, l.cuda(), 4, score="sigmoid", n_groups=10, keep_groups=2, group_top=2)
    _check(l, l.cuda(), 4, score="softmax", bias=torch.zeros(100), n_groups=10, keep_groups=2, group_top=1)


def test_extreme_logits():
    """Infinities, NaN, the type's lowest and largest values and denormal numbers, in every place of a row."""
    big = torch.finfo(torch.float32).max
    v = [float("inf"), -float("inf"), float("nan"), big, -big, 1e-42, -1e-42, 0.0, 700.0, -700.0, 36.0, 1.0]
    rows = [[v[(i * j + i) % 12] for j in range(12)] for i in range(12)] + [v, v[::-1], [-big] * 12, [big] * 12]
    l = torch.tensor(rows)
    # (a sigmoid of 36 and of 700 are neighbours in binary64: only without a
    # bias, where the logits decide, is their order the formula's)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx, g = _check(l, l.cuda(), 5, score=score, renorm=renorm)
            assert torch.isfinite(g).all()


NANS = {torch.bfloat16: [0x7F81, 0xFF81, 0x7FBF, 0xFFBF, 0x7FC0, 0xFFFF],
        torch.float32: [0x7F800001, 0xFF800001, 0x7FBFFFFF, 0xFFBFFFFF, 0x7FC00000, 0xFFFFFFFF]}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,pitch", [(8, 0), (60, 61), (256, 0)])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_every_kind_of_nan(dtype, E, pitch, score, renorm):
    """Quiet and signalling NaN of either sign, copied as bits, in aligned and unaligned rows: not available."""
    l, _ = _logits(24, E, dtype, 5)
    width = 8 * l.element_size()
    ints = l.view(torch.int16 if width == 16 else torch.int32)
    for n, t in enumerate(range(1, 24)):
        for j in range(3):
            p = NANS[dtype][(3 * n + j) % 6]
            ints[t, (7 * t + 3 * j) % E] = p - (1 << width) if p >> (width - 1) else p
    wide = torch.zeros((24, pitch or E), dtype=ints.dtype, device="cuda")
    wide[:, :E] = ints.cuda()
    idx, _ = _check(l, wide.view(dtype)[:, :E], 4, score=score, renorm=renorm)
    took = l.gather(1, idx.cpu().clamp(min=0).long())
    assert not took[idx.cpu() >= 0].isnan().any()


def test_every_bf16_logit():
    """All 65536 bit patterns as logits, 256 neighbouring ones a row."""
    ints = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(256, 256)
    for score in ("softmax", "sigmoid"):
        _check(ints.view(torch.bfloat16), ints.cuda().view(torch.bfloat16), 8, score=score, renorm=False)


def test_bias_that_excludes():
    """-inf and NaN in the bias make an expert unavailable to be chosen, +inf puts it first; the weights do not know the bias."""
    l, dev = _logits(40, 16, torch.float32, 4)
    bias = torch.zeros(16)
    bias[3] = float("inf")
    bias[5] = -float("inf")
    bias[6] = float("nan")
    idx, g = dlm.route(dev, 15, bias=bias.cuda(), renorm=False)
    s, _ = ref.scores(l.double().numpy(), "softmax")
    i = idx.cpu().numpy()
    assert (i[:, 0] == 3).all() and not np.isin(i, [5, 6]).any() and (i[:, 14] == -1).all()
    want = np.take_along_axis(s, i[:, :14], 1)
    assert (np.abs(g.cpu().double().numpy()[:, :14] - want) <= 2.0 ** -24 * want + R64).all()


def test_gradient_against_differences():
    """Central differences of the weights of a fixed choice; the step's error is of second order:
    h^2 / 6 times the third derivative, below 1e-6 * (k * max|dg| * scale) at h = 1e-3."""
    T, E, k = 6, 12, 3
    l, dev = _logits(T, E, torch.float32, 9)
    ln = l.double().numpy()
    dg = np.random.default_rng(0).standard_normal((T, k)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx, _ = dlm.route(dev, k, score=score, renorm=renorm, scale=2.0)
            got = dlm.route_backward(dev, idx, torch.from_numpy(dg).cuda(), score=score, renorm=renorm, scale=2.0)
            i, h = idx.cpu().numpy(), 1e-3
            for e in range(E):
                up, dn = ln.copy(), ln.copy()
                up[:, e] += h
                dn[:, e] -= h
                d = (ref.weights(up, i, score, renorm, 2.0) - ref.weights(dn, i, score, renorm, 2.0)) * dg
                want = d.sum(1) / (2 * h)
                assert np.abs(got[:, e].cpu().double().numpy() - want).max() <= 2e-6 * k * np.abs(dg).max()


def test_backward_of_any_choice():
    """A choice that dlm.route did not make: an expert twice, empty slots, indices outside, an unavailable expert."""
    l, dev = _logits(6, 20, torch.float32, 1)
    l[5, 4] = -float("inf")
    dev = l.cuda()
    idx = torch.tensor([[3, 3, 7], [-1, 2, -1], [-1, -1, -1], [20, 1, -5], [19, 0, 19], [4, 5, 6]], dtype=torch.int32)
    dg = torch.randn((6, 3), generator=torch.Generator().manual_seed(0))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = dlm.route_backward(dev, idx.cuda(), dg.cuda(), score=score, renorm=renorm).cpu().double().numpy()
            want = ref.route_backward(l.double().numpy(), idx.numpy(), dg.double().numpy(), score, renorm)
            assert (np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + R64 * 32).all()


def test_streams_and_graph():
    """On another stream and replayed from a graph, with eager work between the replays: the eager bits."""
    l, dev = _logits(300, 64, torch.float32, 8)
    dg = torch.randn((300, 4), generator=torch.Generator().manual_seed(0)).cuda()
    want = dlm.route(dev, 4)
    wantd = dlm.route_backward(dev, want[0], dg)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    i2, g2 = dlm.route(dev, 4, stream=s)
    s.synchronize()
    assert torch.equal(i2, want[0]) and torch.equal(g2, want[1])
    idx, g = torch.empty_like(want[0]), torch.empty_like(want[1])
    dl, counts = torch.empty_like(wantd), torch.zeros(64, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dlm.route(dev, 4, idx=idx, g=g, counts=counts)
        dlm.route_backward(dev, idx, dg, dlogits=dl)
    for r in range(3):
        idx.fill_(-9)
        dl.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, want[0]) and torch.equal(g, want[1]) and torch.equal(dl, wantd)
        assert int(counts.sum()) == 300 * 4 * (r + 1)


def test_the_chosen_sets_feed_the_sgmm():
    """k = 2: idx and g are the per-row sets the SGMM takes; the bare top 2 is dlm.pregate's choice."""
    T, d, E = 50, 64, 8
    gen = torch.Generator().manual_seed(0)
    x = torch.randn((T, d), generator=gen).cuda()
    Wr = (torch.randn((d, E), generator=gen) * 0.02).cuda()
    logits = (x.double() @ Wr.double()).float()
    idx, g = dlm.route(logits, 2)
    pi, pg = dlm.pregate(x, Wr)
    assert torch.equal(idx, pi)
    # both weights are functions of the logits' difference, which fp32 logits hold to 2^-24 of their size
    assert (g - pg).abs().max().item() <= 2.0 ** -23 * max(1.0, logits.abs().max().item())


def test_empty_batch():
    l = torch.empty((0, 8), device="cuda")
    idx, g = dlm.route(l, 2)
    assert idx.shape == (0, 2) and dlm.route_backward(l, idx, g).shape == (0, 8)


def test_refusals_of_the_binding():
    l = torch.zeros((4, 8), device="cuda")
    for kw in ({"k": 0}, {"k": 9}, {"k": 17}, {"k": 2, "n_groups": 3}, {"k": 5, "n_groups": 4, "keep_groups": 2},
               {"k": 2, "keep_groups": 2}, {"k": 2, "group_top": 3}, {"k": 2, "scale": float("nan")}):
        with pytest.raises(dlm.DLMError):
            dlm.route(l, **kw)
    with pytest.raises(ValueError):
        dlm.route(l, 2, score="tanh")
    with pytest.raises(ValueError):
        dlm.route(l.t(), 2)
    with pytest.raises(ValueError):
        dlm.route(l[:1].expand(4, 8), 2)
    with pytest.raises(ValueError):
        dlm.route(l.cpu(), 2)
    with pytest.raises(ValueError):
        dlm.route(l, 2, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        dlm.route(l, 2, counts=torch.zeros(8, device="cuda"))
    with pytest.raises(TypeError):
        dlm.route(l.half(), 2)
    with pytest.raises(dlm.DLMError):
        dlm.route_backward(l, torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda"),
                           dlogits=l)
