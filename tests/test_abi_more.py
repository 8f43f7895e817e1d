"""Refusals of the balance loss on the host before any HIP call (no GPU: every call below fails
validation or has nothing to do), and the plain forms of the tests against differences."""
import ctypes as C
import os

import pytest
import torch

import balance_ref
import dynamic_lora_moe_amd as dlm

P = C.c_void_p
FAKE = 0x100000
MB = 1 << 20

built = pytest.mark.skipif(not os.path.exists(dlm.LIB_PATH), reason="libdlm.so not built")


@built
def test_balance_validation():
    lib = dlm.load()
    b = C.c_size_t(0)
    size = lib.dlm_balance_workspace_size
    assert size(4, 8, 1, None) == dlm.DLM_EINVAL
    for T, E, S in ((-1, 8, 1), (1 << 31, 8, 1), (4, 0, 1), (4, 513, 1), (4, 8, 0), (4, 8, 65537)):
        assert size(T, E, S, C.byref(b)) == dlm.DLM_ESHAPE
    assert size(4, 8, 3, C.byref(b)) == dlm.DLM_OK and b.value > 0
    at = [FAKE + k * 64 * MB for k in range(12)]

    def cfg(k=2, score=0, alpha=0.1, zeta=0.0):
        return C.byref(dlm.dlm_balance_cfg(k, score, alpha, zeta))

    def fwd(logits=at[0], ld=8, idx=at[1], off=None, S=1, T=4, E=8, dt=0, c=None, loss=at[2], counts=at[3], rows=at[4],
            probs=at[5], ws=at[6], wb=64 * MB):
        return lib.dlm_balance(P(logits), ld, P(idx), P(off), S, T, E, dt, c or cfg(), P(loss), P(counts), P(rows), P(probs), P(ws),
                               wb, None)

    def bwd(logits=at[0], ld=8, counts=at[3], rows=at[4], off=None, S=1, T=4, E=8, dt=0, c=None, dloss=None, dl=at[7], ldd=8):
        return lib.dlm_balance_backward(P(logits), ld, P(counts), P(rows), P(off), S, T, E, dt, c or cfg(), P(dloss), 0, P(dl), ldd,
                                        None)

    for f in (fwd, bwd):
        assert f(T=-1) == dlm.DLM_ESHAPE and f(T=1 << 31) == dlm.DLM_ESHAPE
        assert f(E=0) == dlm.DLM_ESHAPE and f(E=513, ld=513) == dlm.DLM_ESHAPE and f(ld=7) == dlm.DLM_ESHAPE
        assert f(S=0) == dlm.DLM_ESHAPE and f(S=65537, off=at[8]) == dlm.DLM_ESHAPE
        assert f(S=2) == dlm.DLM_EINVAL  # no offsets
        assert f(dt=2) == dlm.DLM_EDTYPE
        assert f(logits=None) == dlm.DLM_EINVAL and f(counts=None) == dlm.DLM_EINVAL and f(rows=None) == dlm.DLM_EINVAL
        assert f(c=cfg(k=0)) == dlm.DLM_ESHAPE and f(c=cfg(k=17)) == dlm.DLM_ESHAPE
        assert f(c=cfg(score=2)) == dlm.DLM_EINVAL
        assert f(c=cfg(alpha=float("inf"))) == dlm.DLM_EINVAL and f(c=cfg(zeta=float("nan"))) == dlm.DLM_EINVAL
        assert f(c=cfg(score=1, zeta=0.1)) == dlm.DLM_EINVAL
        assert f(logits=at[0] + 2) == dlm.DLM_EALIGN and f(counts=at[3] + 1) == dlm.DLM_EALIGN
        assert f(off=at[8] + 2) == dlm.DLM_EALIGN
    assert lib.dlm_balance(P(at[0]), 8, P(at[1]), None, 1, 4, 8, 0, None, P(at[2]), P(at[3]), P(at[4]), P(at[5]), P(at[6]), MB,
                           None) == dlm.DLM_EINVAL
    for k in ("idx", "loss", "probs"):
        assert fwd(**{k: None}) == dlm.DLM_EINVAL
    assert fwd(ws=None) == dlm.DLM_EWORKSPACE and fwd(wb=16) == dlm.DLM_EWORKSPACE and fwd(ws=at[6] + 8) == dlm.DLM_EALIGN
    # written buffers overlap nothing
    for k in ("loss", "counts", "rows", "probs", "ws"):
        assert fwd(**{k: at[0]}) == dlm.DLM_EINVAL and fwd(**{k: at[1]}) == dlm.DLM_EINVAL
    assert fwd(off=at[3]) == dlm.DLM_EINVAL and fwd(rows=at[3]) == dlm.DLM_EINVAL
    assert bwd(dl=None) == dlm.DLM_EINVAL and bwd(ldd=7) == dlm.DLM_ESHAPE
    for k in (0, 3, 4):
        assert bwd(dl=at[k]) == dlm.DLM_EINVAL
    assert bwd(dl=at[8], dloss=at[8]) == dlm.DLM_EINVAL
    assert bwd(T=0, logits=None, counts=None, rows=None, dl=None) == dlm.DLM_OK


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_is_the_loss_derivative(score):
    """The plain gradient against central differences of the plain loss, in binary64, the counts held."""
    gen = torch.Generator().manual_seed(1)
    T, E, k, off = 12, 5, 2, [1, 4, 4, 11]
    l = torch.randn((T, E), generator=gen, dtype=torch.float64)
    l[2, 3] = -float("inf")
    l[5] = -float("inf")
    idx = torch.randint(0, E, (T, k), generator=gen)
    zeta = 0.3 if score == "softmax" else 0.0
    _, counts, rows, _ = balance_ref.balance(l, idx, score, 0.7, zeta, off)
    dl, _ = balance_ref.backward(l, counts, rows, k, score, 0.7, zeta, off, (2.0, 3.0))
    assert counts.sum() == sum(int(l[t, e] > -float("inf")) for t in range(1, 11) for e in idx[t].tolist())
    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, dn = l.clone(), l.clone()
            up[t, e] += h
            dn[t, e] -= h
            a, b = (balance_ref.balance(v, idx, score, 0.7, zeta, off)[0] for v in (up, dn))
            want = float((2 * (a[0] - b[0]) + 3 * (a[1] - b[1])) / (2 * h))
            # differences: h^2 of truncation, 2^-52 / h of rounding
            assert abs(float(dl[t, e]) - want) < 1e-8, (t, e)


def test_balance_by_hand():
    l = torch.log(torch.tensor([[1.0, 3.0], [1.0, 1.0]]))
    loss, counts, rows, probs = balance_ref.balance(l, torch.tensor([[1], [0]]), "softmax", 1.0, 1.0)
    assert counts.tolist() == [[1, 1]] and rows.tolist() == [2]
    assert torch.allclose(probs, torch.tensor([[0.375, 0.625]], dtype=torch.float64))
    assert abs(float(loss[0]) - 1.0) < 1e-6  # f = (1, 1)
    assert abs(float(loss[1]) - (torch.log(torch.tensor(4.0)) ** 2 + torch.log(torch.tensor(2.0)) ** 2) / 2) < 1e-6


def _muon_params(*ps):
    arr = (dlm.dlm_muon_param * len(ps))()
    for i, p in enumerate(ps):
        arr[i] = dlm.dlm_muon_param(*p)
    return arr


@built
def test_muon_validation():
    lib = dlm.load()
    h = C.c_void_p()
    a = [FAKE + k * MB for k in range(8)]
    fine = (a[0], a[1], None, a[2], 2, 5, 10, 0.01, 1.0)

    def create(ps, n=1, pd=0, gd=0, out=True):
        return lib.dlm_muon_create(ps, n, pd, gd, C.byref(h) if out else None)

    def put(**kw):
        names = ("p", "g", "master", "m", "count", "rows", "cols", "wd", "scale")
        return _muon_params(tuple(kw.get(k, v) for k, v in zip(names, fine)))

    assert create(None) == dlm.DLM_EINVAL and create(put(), 0) == dlm.DLM_EINVAL and create(put(), out=False) == dlm.DLM_EINVAL
    assert create(put(), pd=3) == dlm.DLM_EDTYPE and create(put(), gd=-1) == dlm.DLM_EDTYPE
    for k in ("p", "g", "m"):
        assert create(put(**{k: None})) == dlm.DLM_EINVAL
    for k, v in (("rows", 0), ("cols", 0), ("count", -1), ("rows", 1 << 31), ("cols", -5)):
        assert create(put(**{k: v})) == dlm.DLM_ESHAPE
    assert create(put(rows=513, cols=600)) == dlm.DLM_ESHAPE
    assert create(put(count=1 << 29, rows=512, cols=1 << 29)) == dlm.DLM_ESHAPE
    assert create(put(wd=float("nan"))) == dlm.DLM_EINVAL and create(put(scale=float("inf"))) == dlm.DLM_EINVAL
    assert create(put(master=a[3])) == dlm.DLM_EINVAL  # an fp32 parameter has none
    assert create(put(p=a[0] + 2)) == dlm.DLM_EALIGN and create(put(p=a[0] + 1), pd=1) == dlm.DLM_EALIGN
    assert create(put(m=a[2] + 1)) == dlm.DLM_EALIGN
    assert create(put(g=a[0])) == dlm.DLM_EINVAL and create(put(m=a[1])) == dlm.DLM_EINVAL
    other = (a[4], a[1] + 100, None, a[2] + 396, 1, 5, 10, 0.0, 1.0)
    assert create(_muon_params(fine, other), 2) == dlm.DLM_EINVAL and "1" in lib.dlm_last_error().decode()
    assert h.value is None
    cfg = dlm.dlm_muon_cfg(1e-3, 0.95, 1, 1e-7, 5)
    assert lib.dlm_muon_step(None, C.byref(cfg), None, None, None) == dlm.DLM_EINVAL
    assert lib.dlm_muon_destroy(None) == dlm.DLM_EINVAL and lib.dlm_muon_status(None, None, None) == dlm.DLM_EINVAL


@built
@pytest.mark.parametrize("count, rows, cols", [(1 << 30, 2, 2), (1 << 25, 16, 40), (1 << 24, 40, 33), (1 << 20, 65, 65), (300000, 512, 512),
                                               (1 << 15, 128, 1 << 17), (1, 65, 1 << 30)])
def test_muon_grids(count, rows, cols):
    """More pieces, matrices or products than a launch can hold are refused, before tables are made for them."""
    import time

    h, tb = C.c_void_p(), 1 << 44
    start = time.perf_counter()
    rc = dlm.load().dlm_muon_create(_muon_params((tb, 2 * tb, None, 3 * tb, count, rows, cols, 0.0, 1.0)), 1, 0, 0, C.byref(h))
    assert rc == dlm.DLM_ESHAPE and h.value is None
    assert time.perf_counter() - start < 2


@pytest.mark.parametrize("shape", [(3, 8), (8, 3), (5, 5)])
def test_muon_by_values_is_muon_by_products(shape):
    import muon_ref
    import numpy as np

    u = np.random.default_rng(0).standard_normal(shape)
    c = [muon_ref.COEFS] * 5
    assert np.abs(muon_ref.by_values(u, 1e-7, c) - muon_ref.by_products(u, 1e-7, c)).max() < 1e-12
    assert np.abs(muon_ref.by_products(u, 1e-7, c) - muon_ref.by_products(u.T, 1e-7, c).T).max() < 1e-12


@built
def test_int8_validation():
    lib = dlm.load()
    h = C.c_void_p()
    a = [FAKE + k * 64 * MB for k in range(8)]

    def create(n=1, dt=0, out=True, **kw):
        v = dict(x=a[0], W=a[1], w_scale=a[2], y=a[3], d_in=32, d_out=8) | kw
        return lib.dlm_i8_group_create((dlm.dlm_i8_problem * 1)(dlm.dlm_i8_problem(*v.values())), n, dt, C.byref(h) if out else None)

    assert lib.dlm_i8_group_create(None, 1, 0, C.byref(h)) == dlm.DLM_EINVAL
    assert create(n=0) == dlm.DLM_EINVAL and create(n=65536) == dlm.DLM_EINVAL and create(out=False) == dlm.DLM_EINVAL
    assert create(dt=2) == dlm.DLM_EDTYPE
    for k in ("x", "W", "w_scale", "y"):
        assert create(**{k: None}) == dlm.DLM_EINVAL
    for d in (0, -1, 131073):
        assert create(d_in=d) == dlm.DLM_ESHAPE
    assert create(d_out=0) == dlm.DLM_ESHAPE and create(d_out=1 << 31) == dlm.DLM_ESHAPE
    assert create(x=a[0] + 2) == dlm.DLM_EALIGN and create(y=a[3] + 1, dt=1) == dlm.DLM_EALIGN and create(w_scale=a[2] + 2) == dlm.DLM_EALIGN
    assert h.value is None
    b = C.c_size_t(0)
    assert lib.dlm_i8_group_workspace_size(None, 4, C.byref(b)) == dlm.DLM_EINVAL
    assert lib.dlm_i8_group_backward_workspace_size(None, 4, C.byref(b)) == dlm.DLM_EINVAL
    assert lib.dlm_i8_group_run(None, 4, P(a[4]), MB, None) == dlm.DLM_EINVAL
    assert lib.dlm_i8_group_backward(None, 4, 0, P(a[4]), MB, None) == dlm.DLM_EINVAL
    assert lib.dlm_i8_group_bind_grads(None, None, None) == dlm.DLM_EINVAL
    assert lib.dlm_i8_group_destroy(None) == dlm.DLM_EINVAL
    q = lib.dlm_i8_quantize
    assert q(P(a[0]), -1, 8, 0, P(a[1]), P(a[2]), None) == dlm.DLM_ESHAPE and q(P(a[0]), 4, 0, 0, P(a[1]), P(a[2]), None) == dlm.DLM_ESHAPE
    assert q(P(a[0]), 4, 8, 5, P(a[1]), P(a[2]), None) == dlm.DLM_EDTYPE
    assert q(None, 4, 8, 0, P(a[1]), P(a[2]), None) == dlm.DLM_EINVAL and q(P(a[0]), 4, 8, 0, None, P(a[2]), None) == dlm.DLM_EINVAL
    assert q(P(a[0] + 2), 4, 8, 0, P(a[1]), P(a[2]), None) == dlm.DLM_EALIGN
    assert q(P(a[0]), 4, 8, 0, P(a[0] + 16), P(a[2]), None) == dlm.DLM_EINVAL and q(P(a[0]), 4, 8, 0, P(a[1]), P(a[1]), None) == dlm.DLM_EINVAL
    assert q(None, 0, 8, 0, None, None, None) == dlm.DLM_OK


def test_int8_codes_by_hand():
    import int8_ref

    q, s = int8_ref.codes(torch.tensor([[1.0, 0.5, -0.5, 0.51, 0.0], [0.0, 0.0, 0.0, 0.0, 0.0]]))
    assert q.tolist() == [[127, 63, -63, 65, 0], [0] * 5] and s[1] == 0 and abs(float(s[0]) * 127 - 1) < 1e-6
