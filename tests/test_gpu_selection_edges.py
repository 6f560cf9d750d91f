"""Calls of the selection operators at the ends of their ranges, on the GPU
against the plain 64-bit implementation.  Tolerances are those of
test_gpu_route.py and test_gpu_logits.py, which state how they are made."""
import math

import numpy as np
import pytest

from gpu_util import device, note
from oracle import selection as plain
from test_gpu_logits import (SUM_ERROR, check_pick, gpu_rules, lib, make_logits, make_rules,
                             row_parameters, same, to_gpu)
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


@pytest.mark.parametrize("E,G,kept,k", [(4, 2, 1, 2), (32, 16, 7, 6), (48, 16, 10, 5),
                                        (128, 64, 32, 8), (120, 30, 24, 9), (64, 8, 3, 6),
                                        (256, 8, 4, 8), (512, 128, 60, 8)])
@pytest.mark.parametrize("biased", [False, True])
def test_groups_whose_sums_are_equal(E, G, kept, k, biased):
    """Sigmoid scores of z and of -z sum to 1 for every z: groups of such pairs
    are equal, and the lower ones stay."""
    rng = np.random.default_rng([E, G])
    z = np.round(rng.normal(size=(60, E)) * 2) / 2
    z[:, 1::2] = np.where(rng.random((60, E // 2)) < 0.6, -z[:, ::2], z[:, 1::2])
    z[0, 1::2] = -z[0, ::2]
    for dtype in (torch.float32, torch.bfloat16):
        check_route(torch.from_numpy(z).to(dtype), z, score="sigmoid", top_k=k, groups=G,
                    kept_groups=kept, bias=np.zeros(E, np.float32) if biased else None)


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


@pytest.mark.parametrize("V,k", [(40, 1), (40, 30), (9000, 40), (33000, 400), (70000, 900),
                                 (70000, 1)])
@pytest.mark.parametrize("size", [1e-44, 1e-41, 1e-38])
def test_temperatures_below_the_normal_numbers(V, k, size):
    """Logits of the same size as the temperature, down to its smallest step."""
    rng = np.random.default_rng([V, k])
    z = (rng.normal(size=(4, V)) * size).astype(np.float32)
    z[3, ::3] = -np.inf
    for t in (1e-45, 1e-41, 1e-38):
        check_pick(torch.from_numpy(z), z, "t=%g" % t, uniform=rng.random(4).astype(np.float32),
                   max_top_k=k, temperature=np.full(4, t, np.float32))


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


# --------------------------------------------- rows of more slices and forms

def most_in_late_slices(rng, B, V, crowded=False):
    """bfloat16 values, so that many are equal; the largest in the last slices."""
    z = torch.from_numpy(rng.normal(size=(B, V)).astype(np.float32))
    z[0, V - V // 16:] += 3.0
    if crowded:
        z[-1] = torch.round(z[-1])
        z[-1, -9:] = z[-1].max()
    return z.bfloat16()


@pytest.mark.parametrize("V", [150001, 262147])
@pytest.mark.parametrize("k", [1000, 1024])
def test_more_candidates_than_a_join_holds(V, k):
    """The join's waves hold 192 pieces of 64 candidates; these rows have 240
    to 425, so that the rest is read again for every pass over them."""
    rng = np.random.default_rng([V, k])
    z = most_in_late_slices(rng, 5, V, crowded=True).float().numpy()
    z[1] = 0.0
    z[2] = np.sort(z[2])
    z[3, rng.random(V) < 0.9] = np.finfo(np.float32).min
    for _ in range(2):
        check_pick(torch.from_numpy(z), z, **row_parameters(rng, 5, k))
        check_pick(torch.from_numpy(z), z, uniform=rng.random(5).astype(np.float32), max_top_k=k,
                   temperature=np.full(5, 3.0, np.float32))


@pytest.mark.parametrize("V", [1048577, 1100003, 4194304])
@pytest.mark.parametrize("k", [1, 40, 1024])
def test_more_slices_than_a_wave_has_lanes(V, k):
    rng = np.random.default_rng([V, k])
    z = most_in_late_slices(rng, 3, V, crowded=True)
    zf = z.float().numpy()
    check_pick(z, zf, **row_parameters(rng, 3, k))
    zf = np.full((2, V), -np.inf, np.float32)
    zf[0, -1] = 1.0
    zf[1, V - 30000:] = rng.normal(size=30000)
    check_pick(torch.from_numpy(zf), zf, uniform=rng.random(2).astype(np.float32), max_top_k=k)
    u = make_rules(rng, 3, V, L=500)
    check_pick(z, plain.adjust(z.float().numpy(), **u), rules=gpu_rules(V, u),
               **row_parameters(rng, 3, k))


@pytest.mark.parametrize("V", [700, 8192, 8193])
@pytest.mark.parametrize("k", [1, 40, 600])
@pytest.mark.parametrize("B", [256, 257, 300])
def test_many_short_rows(B, V, k):
    """Both sides of the border between one launch and two, and of that between
    slices of 8192 and of 16384."""
    rng = np.random.default_rng([B, V, k])
    z = most_in_late_slices(rng, B, V, crowded=True)
    zf = z.float().numpy()
    check_pick(z, zf, **row_parameters(rng, B, k))


@pytest.mark.parametrize("V", [16384, 16385, 32767, 32768, 32769])
@pytest.mark.parametrize("k", [1, 256, 257])
def test_borders_of_a_row_in_one_launch(V, k):
    rng = np.random.default_rng([V, k])
    z = most_in_late_slices(rng, 4, V, crowded=True)
    u = make_rules(rng, 4, V, L=500)
    check_pick(z, plain.adjust(z.float().numpy(), **u), rules=gpu_rules(V, u),
               **row_parameters(rng, 4, k))


@pytest.mark.parametrize("B,V", [(256, 16384), (255, 16384), (64, 8192), (63, 8192), (2, 4194304),
                                 (40, 40000)])
@pytest.mark.parametrize("L", [4096, 4097])
def test_borders_of_adjusting(B, V, L):
    rng = np.random.default_rng([B, V, L])
    u = make_rules(rng, B, V, L)
    z, zf = make_logits(rng, B, V, "bf16")
    note("adjust %d %d %d" % (B, V, L))
    same(lib().adjust_logits(z.to(device()), gpu_rules(V, u)), plain.adjust(zf, **u))


# ----------------------------------------------------- rules whose tensors move

def test_rules_of_a_history_that_grows():
    rng = np.random.default_rng(31)
    B, V = 3, 900
    z, zf = make_logits(rng, B, V, "f32")
    z = z.to(device())
    u = make_rules(rng, B, V, L=10)
    on = {k: to_gpu(v) for k, v in u.items()}
    rules = lib().LogitRules(V, **on)
    same(lib().adjust_logits(z, rules), plain.adjust(zf, **u))
    for L in (200, 7, 5000, 5001):
        u.update({k: v for k, v in make_rules(rng, B, V, L=L).items() if "len" in k or
                  k == "history"})
        on["history"].resize_(B, L)
        for name in ("history", "history_len", "prompt_len"):
            on[name].copy_(to_gpu(u[name]))
        same(lib().adjust_logits(z, rules), plain.adjust(zf, **u))
        check_pick(z, plain.adjust(zf, **u), rules=rules, **row_parameters(rng, B, 20))
    u["repetition"] = np.full(B, 1.75, np.float32)
    on["repetition"].data = to_gpu(u["repetition"])
    u["allowed"] = rng.integers(-2 ** 63, 2 ** 63 - 1, size=(4, 20), dtype=np.int64)
    on["allowed"].set_(to_gpu(u["allowed"]))
    same(lib().adjust_logits(z, rules), plain.adjust(zf, **u))


def test_an_empty_batch_with_rules():
    u = make_rules(np.random.default_rng(32), 3, 100)
    on = {k: to_gpu(v)[:0] if k != "allowed" else to_gpu(v) for k, v in u.items()}
    rules = lib().LogitRules(100, **on)
    z = torch.zeros(0, 100, device=device())
    assert lib().adjust_logits(z, rules).shape == (0, 100)
    ids, lp = lib().pick_tokens(z, torch.zeros(0, device=device()), rules=rules)
    assert ids.shape == (0,) and lp.shape == (0,)


def test_picking_and_nms_in_turn():
    """Both keep a workspace per thread and stream."""
    g = lib()
    rng = np.random.default_rng(33)
    n = 3000
    at = rng.random((n, 2)).astype(np.float32) * 300
    boxes = torch.from_numpy(np.concatenate([at, at + 1 + rng.random((n, 2)).astype(np.float32)
                                             * 30], axis=1)).to(device())
    scores = torch.from_numpy(rng.random(n).astype(np.float32)).to(device())
    z, zf = make_logits(rng, 4, 70000, "f32")
    first = g.nms(boxes, scores, 0.5)
    for _ in range(4):
        check_pick(z, zf, **row_parameters(rng, 4, 900))
        assert torch.equal(g.nms(boxes, scores, 0.5), first)


# ------------------------------------------ neighbours that must not matter

# Logits of a token's chosen experts one of whose weights rounds to another
# float32 by a quotient than by the product with an inverse.
CHOSEN = [
    ("sigmoid", ["0x1.9407aap+1", "0x1.61eeaap+1", "0x1.12773ep+1", "0x1.7f0f08p+0",
                 "0x1.6d8c74p+0", "0x1.6a6820p+0", "0x1.43f9d8p+0", "0x1.3fc452p+0"]),
    ("sigmoid", ["0x1.14e26ap+1", "0x1.ac24a0p+0", "0x1.906c46p+0", "0x1.7461ccp+0",
                 "0x1.5e7af0p+0", "0x1.4ec740p+0", "0x1.4a7b12p+0", "0x1.309752p+0"]),
    ("sigmoid", ["0x1.0f36bap+1", "0x1.0027c8p+1", "0x1.da1202p+0", "0x1.c05c2ap+0",
                 "0x1.9ea182p+0", "0x1.83a776p+0", "0x1.82e9f0p+0", "0x1.5de654p+0"]),
    ("sigmoid", ["0x1.c8b170p+0", "0x1.c357f6p+0", "0x1.9d2024p+0", "0x1.5896cep+0",
                 "0x1.1cea1ap+0", "0x1.be1084p-1", "0x1.a3ec4ap-1", "0x1.9ed144p-1"]),
    ("sigmoid", ["0x1.3102c0p+1", "0x1.eeb8bap+0", "0x1.ee3de8p+0", "0x1.c11f76p+0",
                 "0x1.bc5598p+0", "0x1.b2df18p+0", "0x1.4794cap+0", "0x1.2843c2p+0"]),
    ("softmax", ["0x1.46891cp+1", "0x1.fd7e7ap+0", "0x1.f5639ep+0", "0x1.e9c392p+0",
                 "0x1.e5dc32p+0", "0x1.7e87cep+0", "0x1.66a43ap+0", "0x1.38acb8p+0"]),
]


@pytest.mark.parametrize("score,chosen", CHOSEN)
@pytest.mark.parametrize("E", [8, 64, 200, 500])
def test_weights_do_not_depend_on_padded_neighbours(E, score, chosen):
    rng = np.random.default_rng(E)
    dev = device()
    z = np.full((9, E), -40.0, np.float32)
    z[:, rng.permutation(E)[:8]] = [float.fromhex(x) for x in chosen]
    z = torch.from_numpy(z).to(dev)
    ids, w = lib().route_experts(z, 8, score=score)
    live = torch.ones(9, dtype=torch.bool, device=dev)
    for dead in ([1], [0, 3, 4], [8], list(range(1, 9))):
        live.fill_(True)
        live[dead] = False
        ids1, w1 = lib().route_experts(z, 8, score=score, live=live)
        assert torch.equal(ids1[live], ids[live]) and torch.equal(w1[live], w[live])
    empty = z.clone()
    empty[2] = -math.inf
    _, w1 = lib().route_experts(empty, 8, score=score)
    assert torch.equal(w1[[0, 1, 3]], w[[0, 1, 3]])
