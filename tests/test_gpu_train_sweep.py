"""Random valid configurations of the training operators from fixed seeds, held to
the same checks and bounds as the chosen ones."""
import random

import pytest
import torch

from test_gpu_adamw import TYPES, _run
from test_gpu_route import _check, _logits
from test_gpu_sgmm_grad import BF, F32, Case

pytestmark = pytest.mark.gpu


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


@pytest.mark.parametrize("seed", range(40))
def test_routing(seed):
    rng = random.Random(1000 + seed)
    groups = rng.choice([1, 1, 2, 3, 4, 8, 16, 32])
    E = groups * rng.randint(1, 512 // groups)
    keep = rng.randint(1, groups)
    k = rng.randint(1, min(16, keep * (E // groups)))
    T, dtype = _log(rng, 1, 3000), rng.choice([torch.float32, torch.bfloat16])
    kw = dict(score=rng.choice(["softmax", "sigmoid"]), n_groups=groups, keep_groups=keep, group_top=rng.choice([1, 2]),
              renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5, 0.25]))
    print(T, E, k, dtype, kw, flush=True)
    l, dev = _logits(T, E, dtype, seed, masked=rng.choice([0.0, 0.0, 0.2]), pitch=rng.choice([0, 0, E + rng.randint(0, 9)]))
    bias = torch.randn(E, generator=torch.Generator().manual_seed(seed)) * 0.2 if rng.random() < 0.5 else None
    _check(l, dev, k, bias=bias, seed=seed, **kw)


@pytest.mark.parametrize("seed", range(40))
def test_sgmm_gradients(seed):
    rng = random.Random(2000 + seed)
    bf = rng.random() < 0.8
    n, E = rng.randint(1, 3), rng.randint(1, 32)
    r = rng.randint(1, 128) if bf else rng.randint(1, 12)
    w = 8 if bf else 1
    shapes = [(w * _log(rng, 1, 3000 // w), w * _log(rng, 1, 3000 // w)) for _ in range(n)]
    T = _log(rng, 1, 1500 if E * r > 256 else 3000)
    print(T, shapes, E, r, bf, flush=True)
    c = Case(T, shapes, E, r, BF if bf else F32, seed=seed, scale=rng.choice([0.5, 1.0, 2.0]), rows=T + rng.choice([0, 3]),
             empty=rng.choice([0.0, 0.1, 0.5]), both=rng.choice([0.0, 0.3]), dup=rng.choice([0.0, 0.5])).bind()
    c.run(T=T)
    c.check()


@pytest.mark.parametrize("seed", range(16))
def test_adamw(seed):
    rng = random.Random(3000 + seed)
    p, g, master = rng.choice(TYPES)
    sizes = [_log(rng, 1, 30000) for _ in range(rng.randint(1, 9))]
    bits, shift, step0 = rng.choice([32, 8]), rng.randint(0, 5), rng.choice([0, 7, 5000])
    print(sizes, p, g, master, bits, shift, step0, flush=True)
    _run(sizes, p, g, master, bits, steps=2, shift=shift, step0=step0, seed=seed)
