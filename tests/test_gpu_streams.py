"""Calls on another stream than the current one whose outputs or workspace the binding
makes itself: the allocator hands out memory that work queued on the current stream may
still use, so the launch comes behind that work."""
import time

import pytest
import torch

import dynamic_lora_moe_amd as dlm

pytestmark = pytest.mark.gpu

T, E = 50000, 16


def _rnd(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).cuda()


def _outputs(name):
    """f(stream) -> the tensors that the call makes."""
    logits = _rnd(T, E)
    if name == "route":
        return lambda s: dlm.route(logits, 8, stream=s)
    if name == "route_backward":
        idx, dg = dlm.route(logits, 8)[0], _rnd(T, 8, seed=1)
        return lambda s: (dlm.route_backward(logits, idx, dg, stream=s),)
    if name == "pregate":
        x, W = _rnd(T, 64), _rnd(64, E, seed=1)
        return lambda s: dlm.pregate(x, W, stream=s)
    if name == "pregate_centroid":
        x, C = _rnd(T, 64), _rnd(E, 2, 64, seed=1)
        return lambda s: dlm.pregate_centroid(x, C, stream=s)
    n = 256 * 4000
    m, v = torch.ones(n, dtype=torch.int8, device="cuda"), torch.ones(n, dtype=torch.uint8, device="cuda")
    return lambda s: dlm.adamw_read_state(m, v, torch.ones(4000, device="cuda"), torch.ones(4000, device="cuda"), stream=s)


@pytest.mark.parametrize("name", ["route", "route_backward", "pregate", "pregate_centroid", "adamw_read_state"])
def test_outputs_in_memory_that_is_still_written(name):
    call = _outputs(name)
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = [torch.empty_like(t) for t in want]
    places = {t.data_ptr() for t in old}
    torch.cuda._sleep(100_000_000)
    for t in old:
        t.fill_(77)
    del old, t
    got = call(s)
    assert {t.data_ptr() for t in got} & places  # else nothing was put to the test
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["run", "backward"])
def test_a_workspace_waits_for_its_memory(name):
    """The launch is not over while work queued before on the current stream, which may hold the
    workspace's memory, has not run.  (On several streams: one that shares the current one's hardware
    queue would wait in any case.)"""
    x, A, B = _rnd(300, 64), _rnd(4, 8, 64, seed=1), _rnd(4, 64, 8, seed=2)
    y, dy, dx = _rnd(300, 64, seed=3), _rnd(300, 64, seed=4), torch.zeros_like(x)
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    idx, g = dlm.route(_rnd(300, 4, seed=5), 2)
    grp = dlm.SgmmGroup([(x, A, B, y)], 4, 8, 1.0)
    grp.bind_grads([dy], [dx], [dA], [dB])
    call = grp.run if name == "run" else grp.backward
    call(idx, g)
    torch.cuda.synchronize()
    for s in [torch.cuda.Stream() for _ in range(4)]:
        torch.cuda._sleep(500_000_000)
        workspace = call(idx, g, stream=s)
        done = torch.cuda.Event()
        done.record(s)
        time.sleep(0.02)
        assert not done.query()
        torch.cuda.synchronize()
        assert dlm.sgmm_status(workspace) == dlm.DLM_OK


@pytest.mark.parametrize("bits", [32, 8])
def test_moments_made_on_another_stream_than_the_steps(bits):
    """Zero moments made behind queued work are zero before the handle's first step, on whatever stream."""
    w, g = _rnd(100000), _rnd(100000, seed=1)
    a, b = w.clone(), w.clone()
    want = dlm.AdamW([a], [g], state_bits=bits)
    want.step(1e-3)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(one):
        torch.cuda._sleep(100_000_000)
        opt = dlm.AdamW([b], [g], state_bits=bits)
    opt.step(1e-3, stream=two)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    assert all(torch.equal(x, y) for x, y in zip(opt.states[0], want.states[0]))
