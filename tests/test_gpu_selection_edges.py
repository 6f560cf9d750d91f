"""Calls of the selection operators at the ends of their ranges, on the GPU
against the plain 64-bit implementation.  Tolerances are those of
test_gpu_route.py and test_gpu_logits.py, which state how they are made."""
import math

import numpy as np
import pytest

from gpu_util import device, note
from test_gpu_logits import SUM_ERROR, check_pick, lib, to_gpu
from test_gpu_route import check_route

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# -------------------------------------------------- scores near binary64's end

@pytest.mark.parametrize("E,G,kept", [(16, 1, 1), (16, 4, 3), (300, 1, 1), (1024, 8, 4),
                                      (512, 512, 500), (1000, 200, 150)])
def test_sigmoid_scores_near_the_end_of_binary64(E, G, kept):
    """Scores of 1e-300 to 1e-308 differ in binary64, and from -709.78 down
    they are 0: the choice under a bias is theirs, whichever kernel makes it
    (the last two shapes are those of the kernel that is binary64 throughout)."""
    rng = np.random.default_rng([E, G])
    z = np.linspace(-708.5, -690.5, E)[None].repeat(6, 0)
    z[1] = z[0][::-1]
    z[2] = rng.permutation(z[0])
    z[3, : E // 2] = -720.0
    z[4] = np.where(rng.random(E) < 0.8, -750.0, z[2])
    z[5] = rng.choice([-700.0, -705.0, -691.0], size=E)
    z = z.astype(np.float32)
    for bias in (np.zeros(E, np.float32), np.full(E, 2.0 ** -149, np.float32)):
        check_route(torch.from_numpy(z), z, score="sigmoid", top_k=5, groups=G, kept_groups=kept,
                    group_top=1, bias=bias)


# ------------------------------------------------------ temperatures at the end

@pytest.mark.parametrize("V,k", [(40, 1), (40, 30), (9000, 40), (33000, 400), (70000, 900),
                                 (70000, 1)])
def test_temperatures_that_make_the_largest_distances_small(V, k):
    """Logits that lie further apart than float32 reaches, at temperatures under
    which they weigh nearly alike; masked tokens and NaN among them."""
    rng = np.random.default_rng([V, k])
    low = np.finfo(np.float32).min
    z = rng.normal(size=(6, V)).astype(np.float32)
    z[0, ::2] = low
    z[0, 1] = -low
    z[1] = rng.uniform(-3e38, 3e38, size=V).astype(np.float32)
    z[2] = z[1]
    z[2, ::3] = -np.inf
    z[3] = z[1]
    z[3, 5::7] = np.nan
    z[4] = np.where(np.arange(V) < V // 2, low, -low)
    z[5] = 1e36 * z[5]
    z[5, ::4] = -np.inf
    for t in (np.inf, 3e38, 1e38, 1e37):
        check_pick(torch.from_numpy(z), z, "t=%g" % t, uniform=rng.random(6).astype(np.float32),
                   max_top_k=k, temperature=np.full(6, t, np.float32))


@pytest.mark.parametrize("V,k", [(40, 1), (40, 30), (9000, 40), (33000, 400), (70000, 900)])
def test_infinite_temperature_and_infinite_logits(V, k):
    """All tokens that are allowed weigh alike."""
    rng = np.random.default_rng([V, k])
    z = rng.normal(size=(3, V)).astype(np.float32)
    z[0, 3] = np.inf
    z[1, ::3] = np.inf
    z[1, 1::3] = -np.inf
    z[2, 7] = np.inf
    z[2, ::5] = np.finfo(np.float32).min
    u = np.array([0.0, 0.5, 0.97], np.float32)
    note("pick %s" % ((V, k),))
    ids, lp = lib().pick_tokens(torch.from_numpy(z).to(device()), to_gpu(u), max_top_k=k,
                                temperature=to_gpu(np.full(3, np.inf, np.float32)))
    for b in range(3):
        there = np.flatnonzero(z[b] > -np.inf)
        order = there[np.argsort(-z[b, there], kind="stable")][:k]
        assert int(ids[b]) == order[int(float(u[b]) * len(order))]
        want = -math.log(len(there))
        assert abs(float(lp[b]) - want) <= SUM_ERROR + 2.0 ** -24 * abs(want)
