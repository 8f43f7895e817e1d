"""Refusals of the training operators' entry points, on the host before any HIP
call (no GPU: every call below fails validation or has nothing to do), and the
plain forms of the tests against each other."""
import ctypes as C
import os

import numpy as np
import pytest

import dynamic_lora_moe_amd as dlm
import route_ref

P = C.c_void_p
FAKE = 0x100000
MB = 1 << 20

built = pytest.mark.skipif(not os.path.exists(dlm.LIB_PATH), reason="libdlm.so not built")


def _cfg(**kw):
    c = dict(k=2, score=dlm.DLM_SOFTMAX, n_groups=1, keep_groups=1, group_top=1, renorm=1, scale=1.0)
    c.update(kw)
    return C.byref(dlm.dlm_route_cfg(*[c[f] for f, _ in dlm.dlm_route_cfg._fields_]))


@built
def test_route_validation():
    lib = dlm.load()
    out = P(FAKE + 64 * MB), P(FAKE + 65 * MB)

    def route(logits=P(FAKE), ld=8, bias=None, T=4, E=8, dt=0, cfg=None, idx=out[0], g=out[1], counts=None):
        return lib.dlm_route(logits, ld, bias, T, E, dt, cfg or _cfg(), idx, g, counts, None)

    def back(logits=P(FAKE), ld=8, idx=out[0], dg=out[1], T=4, E=8, dt=0, cfg=None, dl=P(FAKE + 66 * MB), ldd=8):
        return lib.dlm_route_backward(logits, ld, idx, dg, T, E, dt, cfg or _cfg(), dl, ldd, None)

    for f in (route, back):
        assert f(T=-1) == dlm.DLM_ESHAPE and f(T=1 << 31) == dlm.DLM_ESHAPE
        assert f(E=0) == dlm.DLM_ESHAPE and f(E=513, ld=513) == dlm.DLM_ESHAPE
        assert f(ld=7) == dlm.DLM_ESHAPE
        assert f(dt=2) == dlm.DLM_EDTYPE
        assert f(logits=None) == dlm.DLM_EINVAL and f(idx=None) == dlm.DLM_EINVAL
        assert f(cfg=_cfg(score=2)) == dlm.DLM_EINVAL
        assert f(cfg=_cfg(scale=float("inf"))) == dlm.DLM_EINVAL
        assert f(cfg=_cfg(k=0)) == dlm.DLM_ESHAPE and f(cfg=_cfg(k=9)) == dlm.DLM_ESHAPE
        assert f(E=64, ld=64, cfg=_cfg(k=17)) == dlm.DLM_ESHAPE
        assert f(cfg=_cfg(n_groups=3)) == dlm.DLM_ESHAPE and f(cfg=_cfg(n_groups=0)) == dlm.DLM_ESHAPE
        assert f(E=66, ld=66, cfg=_cfg(n_groups=33)) == dlm.DLM_ESHAPE
        assert f(cfg=_cfg(n_groups=4, keep_groups=5)) == dlm.DLM_ESHAPE
        assert f(cfg=_cfg(n_groups=4, keep_groups=0)) == dlm.DLM_ESHAPE
        assert f(cfg=_cfg(k=3, n_groups=4, keep_groups=1)) == dlm.DLM_ESHAPE
        assert f(cfg=_cfg(group_top=0)) == dlm.DLM_EINVAL and f(cfg=_cfg(group_top=3)) == dlm.DLM_EINVAL
        assert f(T=0, logits=None, idx=None) == dlm.DLM_OK
    assert route(g=None) == dlm.DLM_EINVAL
    assert back(dg=None) == dlm.DLM_EINVAL and back(dl=None) == dlm.DLM_EINVAL and back(ldd=7) == dlm.DLM_ESHAPE
    # written buffers overlap nothing
    assert route(idx=P(FAKE)) == dlm.DLM_EINVAL and route(g=out[0]) == dlm.DLM_EINVAL
    assert route(counts=out[0]) == dlm.DLM_EINVAL and route(bias=out[1]) == dlm.DLM_EINVAL
    assert back(dl=P(FAKE)) == dlm.DLM_EINVAL and back(dl=out[1]) == dlm.DLM_EINVAL
    assert lib.dlm_route(P(FAKE), 8, None, 4, 8, 0, None, out[0], out[1], None, None) == dlm.DLM_EINVAL


def test_route_gradient_is_the_weights_derivative():
    """The plain gradient against central differences of the plain weights, in binary64."""
    rng = np.random.default_rng(1)
    l = rng.standard_normal((4, 9))
    l[1, 2] = -np.inf
    dg = rng.standard_normal((4, 3))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx, g = route_ref.route(l, 3, score=score, renorm=renorm, scale=1.5, n_groups=3, keep_groups=2, group_top=2)
            assert np.allclose(g, route_ref.weights(l, idx, score, renorm, 1.5), rtol=1e-13)
            got = route_ref.route_backward(l, idx, dg, score, renorm, 1.5)
            h = 1e-6
            for e in range(9):
                up, dn = l.copy(), l.copy()
                up[:, e] += h
                dn[:, e] -= h
                want = ((route_ref.weights(up, idx, score, renorm, 1.5)
                         - route_ref.weights(dn, idx, score, renorm, 1.5)) * dg).sum(1) / (2 * h)
                # differences: h^2 of truncation, 2^-52 / h of rounding
                assert np.abs(got[:, e] - want).max() < 1e-8


def test_route_plain_form_by_hand():
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    idx, g = route_ref.route(l, 2)
    assert idx.tolist() == [[2, 1]] and np.allclose(g, [[4 / 6, 2 / 6]])
    idx, g = route_ref.route(l, 2, renorm=False)
    assert np.allclose(g, [[0.5, 0.25]])
    idx, g = route_ref.route(l, 2, bias=np.array([1.0, 0, 0, 1.0]))
    assert idx.tolist() == [[0, 3]] and np.allclose(g, [[0.5, 0.5]])
    idx, g = route_ref.route(l, 1, n_groups=2, keep_groups=1, group_top=2)
    assert idx.tolist() == [[2]]


def _params(*ps):
    arr = (dlm.dlm_adamw_param * len(ps))()
    for i, p in enumerate(ps):
        arr[i] = dlm.dlm_adamw_param(*p)
    return arr


@built
def test_adamw_validation():
    lib = dlm.load()
    h = C.c_void_p()
    a = [FAKE + k * MB for k in range(8)]
    ok32 = (a[0], a[1], None, a[2], a[3], None, None, 100, 0.01)
    ok8 = (a[0], a[1], None, a[2], a[3], a[4], a[5], 100, 0.01)

    def create(ps, n=1, pd=0, gd=0, bits=32, step=0, out=True):
        return lib.dlm_adamw_create(ps, n, pd, gd, bits, step, 0, C.byref(h) if out else None)

    assert create(None) == dlm.DLM_EINVAL and create(_params(ok32), 0) == dlm.DLM_EINVAL
    assert create(_params(ok32), out=False) == dlm.DLM_EINVAL
    assert create(_params(ok32), pd=3) == dlm.DLM_EDTYPE and create(_params(ok32), gd=-1) == dlm.DLM_EDTYPE
    assert create(_params(ok32), bits=16) == dlm.DLM_EINVAL
    assert create(_params(ok32), step=-1) == dlm.DLM_EINVAL
    assert create(_params(ok32), bits=8) == dlm.DLM_EINVAL  # no scales
    for k in (0, 1, 3, 4):
        bad = list(ok32)
        bad[k] = None
        assert create(_params(tuple(bad))) == dlm.DLM_EINVAL
    assert create(_params(ok32[:7] + (-1, 0.0))) == dlm.DLM_ESHAPE
    assert create(_params(ok32[:8] + (float("nan"),))) == dlm.DLM_EINVAL
    assert create(_params((a[0], a[1], a[6]) + ok32[3:])) == dlm.DLM_EINVAL  # fp32 parameter with a master
    assert create(_params((a[0] + 2,) + ok32[1:])) == dlm.DLM_EALIGN
    assert create(_params((a[0] + 1,) + ok32[1:]), pd=1) == dlm.DLM_EALIGN
    # buffers that overlap, in one tensor and between two; the second tensor is named
    assert create(_params((a[0], a[0]) + ok32[2:])) == dlm.DLM_EINVAL
    assert create(_params(ok8[:6] + (a[4],) + ok8[7:]), bits=8) == dlm.DLM_EINVAL
    other = (a[6], a[1] + 1000, None, a[2] + 396, a[7], None, None, 100, 0.0)
    assert create(_params(ok32, other), 2) == dlm.DLM_EINVAL
    assert "1" in lib.dlm_last_error().decode()
    assert h.value is None
    cfg = dlm.dlm_adamw_cfg(1e-3, 0.9, 0.999, 1e-8)
    assert lib.dlm_adamw_step(None, C.byref(cfg), None, None, None) == dlm.DLM_EINVAL
    assert lib.dlm_adamw_destroy(None) == dlm.DLM_EINVAL
    assert lib.dlm_adamw_status(None, None, None, None) == dlm.DLM_EINVAL
    rd = lib.dlm_adamw_read_state
    assert rd(a[0], a[1], a[2], a[3], -1, a[4], a[5], None) == dlm.DLM_ESHAPE
    assert rd(None, a[1], a[2], a[3], 5, a[4], a[5], None) == dlm.DLM_EINVAL
    assert rd(a[0], a[1], a[2], a[3], 5, a[4], a[4], None) == dlm.DLM_EINVAL
    assert rd(None, None, None, None, 0, None, None, None) == dlm.DLM_OK


def test_adamw_codes_round_trip():
    """The plain codes: decoding is within one code step, its mean over the noise exact, zeros stay zeros."""
    import adamw_ref

    rng = np.random.default_rng(0)
    m, v = rng.standard_normal(700) * 1e-3, rng.standard_normal(700) ** 2 * 1e-6
    m[:5] = 0
    v[3] = 0
    acc_m, acc_v, n = 0.0, 0.0, 400
    for t in range(n):
        q, c, ms, vs = adamw_ref.encode(m, v, 1, t, 0)
        dm, dv = adamw_ref.decode(q, c, ms, vs)
        b = np.arange(700) // 256
        assert (np.abs(dm - m) <= ms[b] * (2 * np.abs(q.astype(int)) + 1) / 127 ** 2).all()
        assert (dm[:5] == 0).all() and dv[3] == 0 and (dv[v > 0] > 0).all()
        acc_m, acc_v = acc_m + dm, acc_v + dv
    step = ms[b] * (2 * 127 + 1) / 127 ** 2
    assert (np.abs(acc_m / n - m) <= 6 * step / 2 / np.sqrt(n)).all()


@built
def test_backward_validation():
    lib = dlm.load()
    b = C.c_size_t(0)
    assert lib.dlm_sgmm_group_backward_workspace_size(None, 64, C.byref(b)) == dlm.DLM_EINVAL
    assert lib.dlm_sgmm_group_bind_grads(None, None, None, None, None) == dlm.DLM_EINVAL
    assert lib.dlm_sgmm_group_backward(None, P(FAKE), P(FAKE), None, 4, 0, P(FAKE), 1 << 20, None) == dlm.DLM_EINVAL


def test_plain_gradients_against_differences():
    """The plain gradients of the SGMM against differences of the plain product (linear in each argument)."""
    torch = pytest.importorskip("torch")
    import grad_ref

    gen = torch.Generator().manual_seed(0)
    T, E, r, i, o = 7, 3, 2, 5, 4
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, A, B, dy, g = rnd(T, i), rnd(E, r, i), rnd(E, o, r), rnd(T, o), rnd(T, 2)
    idx = torch.tensor([[0, 1], [2, 2], [-1, 0], [-1, -1], [1, -1], [2, 0], [0, 2]])
    (dx, dA, dB, dg), _ = grad_ref.backward(x, idx, g, A, B, dy, 1.5)
    for which, grad in (("x", dx), ("A", dA), ("B", dB), ("g", dg)):
        v = rnd(*grad.shape)
        a = dict(x=x, g=g, A=A, B=B)
        f = lambda s: (grad_ref.forward(**{"idx": idx, "scale": 1.5, **{k: t + s * v if k == which else t for k, t in a.items()}}) * dy).sum()  # noqa: E731
        assert abs(float(f(0.5) - f(-0.5) - (grad * v).sum())) < 1e-10
