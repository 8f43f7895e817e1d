"""The training operators where element offsets pass 2^32, against small calls on
the same values (each row, element or column is worked out for itself)."""
import pytest
import torch

import dynamic_lora_moe_amd as dlm

pytestmark = pytest.mark.gpu


def test_route_past_2_32_logits():
    """More than 2^32 logits: the last rows as a call on them alone gives them."""
    E = 512
    T = (1 << 32) // E + 100
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((150, E), generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    logits[-150:] = tail
    print("route", T, E, flush=True)
    idx, g = dlm.route(logits, 4)
    i2, g2 = dlm.route(tail, 4)
    assert torch.equal(idx[-150:], i2) and torch.equal(g[-150:], g2)
    assert (idx[:-150] == torch.arange(4, device="cuda", dtype=torch.int32)).all()
    dg = torch.zeros_like(g)
    dg[-150:] = torch.randn((150, 4), generator=torch.Generator().manual_seed(1)).cuda()
    dl = dlm.route_backward(logits, idx, dg)
    assert torch.equal(dl[-150:], dlm.route_backward(tail, i2, dg[-150:].contiguous()))
    assert (dl[:-150] == 0).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_past_2_32_elements(bits):
    """One tensor of more than 2^32 elements: elements on both sides of 2^32 and at the end."""
    n, w = (1 << 32) + 5000, 4096
    print("adamw", n, bits, flush=True)
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = [0, (1 << 32) - w, n - n % 256 - w]
    gen = torch.Generator().manual_seed(2)
    vals = [(torch.randn(w, generator=gen).bfloat16().cuda(), (torch.randn(w, generator=gen) * 1e-2).bfloat16().cuda()) for _ in at]
    for a, (pv, gv) in zip(at, vals):
        p[a:a + w], g[a:a + w] = pv, gv
    opt = dlm.AdamW([p], [g], state_bits=bits)
    opt.step(1e-2)
    for a, (pv, gv) in zip(at, vals):
        q = pv.clone()
        small = dlm.AdamW([q], [gv], state_bits=bits)
        small.step(1e-2)
        assert torch.equal(p[a:a + w], q)
        if bits == 32:  # (the 8-bit codes' noise goes by the block's place in its tensor)
            assert all(torch.equal(x[a:a + w], y) for x, y in zip(opt.states[0], small.states[0]))
        else:
            assert torch.equal(opt.states[0][2][a // 256:a // 256 + w // 256], small.states[0][2])
    assert opt.status() == (1, dlm.DLM_OK)


def test_sgmm_gradients_past_2_32_elements():
    """x and dx of more than 2^32 elements: the last rows' dx, and the last columns of dA over all rows."""
    T, d, o, E, r = 66000, 65536, 64, 2, 8
    print("sgmm backward", T, d, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    cols = slice(d - 256, d)
    x[:, cols] = torch.randn((T, 256), generator=gen, device="cuda").bfloat16()
    dx = torch.zeros_like(x)
    A = (torch.randn((E, r, d), generator=gen, device="cuda") * 0.02).bfloat16()
    B = (torch.randn((E, o, r), generator=gen, device="cuda") * 0.2).bfloat16()
    dy = torch.randn((T, o), generator=gen, device="cuda").bfloat16()
    y = torch.empty_like(dy)
    dA, dB = torch.empty(A.shape, device="cuda"), torch.empty(B.shape, device="cuda")
    idx = torch.stack([torch.arange(T, device="cuda") % 2, 1 - torch.arange(T, device="cuda") % 2], 1).int()
    g = torch.rand((T, 2), generator=gen, device="cuda")
    grp = dlm.SgmmGroup([(x, A, B, y)], E, r, 1.0)
    grp.bind_grads([dy], [dx], [dA], [dB])
    dg = torch.empty((T, 2), device="cuda")
    grp.backward(idx, g, dg)
    torch.cuda.synchronize()
    gate = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, idx.long(), g.double())
    w = torch.stack([dy.double() @ B[e].double() for e in range(E)], 1) * gate[:, :, None]  # [T][E][r]
    want = torch.stack([w[:, e].t() @ x[:, cols].double() for e in range(E)])
    # fp32 sums of 2 x 66000 slots over random signs: far inside 2^-14 of the norm, as for small calls
    assert (dA[:, :, cols].double() - want).norm() <= 2.0 ** -14 * want.norm()
    assert (dA[:, :, :d - 256] == 0).all()
    last = (w[-64:].reshape(64, -1) @ A.double().reshape(E * r, d))
    # bf16's rounding, 2^-8 of the value, and the split's 2^-16 of the sum of magnitudes
    mag = w[-64:].abs().reshape(64, -1) @ A.double().abs().reshape(E * r, d)
    assert ((dx[-64:].double() - last).abs() <= 2.0 ** -8 * last.abs() + 2.0 ** -15 * mag).all()
