"""Routing to experts and its gradient on the GPU against the plain 64-bit
implementation.

Tolerances.  ids and counts are whole numbers: equal.  weights: the header
promises 2^-21 of the value (and float32's smallest normal, below which a
value may be 0).  The gradient is computed in float32; with L the row's
largest |z - max z| over eligible experts, a probability is off by at most
(L + 29) 2^-24 of its value (the argument's rounding, 2 ulp of exp, a sum of
at most 22 roundings deep, a quotient), each term of the gradient is a
product of at most two of them and of values with one rounding each, and sums
of k + 6 terms follow: (2 L + 58 + 12 + k) 2^-24 of the sum of the absolute
values of the terms, then half a step of the output's type."""
import math

import numpy as np
import pytest

from gpu_util import device, note
from oracle import selection as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def lib():
    import greedy_iou_nms_amd as g
    return g


def make_logits(rng, T, E, dtype, spread=1.5):
    z = torch.from_numpy(rng.normal(size=(T, E)) * spread).to(DTYPES[dtype])
    return z, z.double().numpy()


def check_route(z, zd, label="", **kw):
    note("route %s %s %s" % (label, tuple(z.shape), kw))
    T, E = z.shape
    dev = device()
    on = {k: (torch.from_numpy(np.asarray(v)).to(dev) if isinstance(v, np.ndarray) else v)
          for k, v in kw.items()}
    got = lib().route_experts(z.to(dev) if not z.is_cuda else z, counts=True, **on)
    ids, w, counts = (t.cpu().numpy() for t in got)
    want_ids, want_w, want_counts = plain.route(zd, **kw)
    np.testing.assert_array_equal(ids, want_ids)
    np.testing.assert_array_equal(counts, want_counts)
    np.testing.assert_allclose(w, want_w, rtol=2.0 ** -21, atol=float(np.finfo(np.float32).tiny))
    return ids


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 7, 7), (5, 16, 4), (64, 60, 4),
                                   (65, 64, 6), (33, 65, 8), (17, 127, 5), (130, 128, 8),
                                   (9, 200, 16), (70, 256, 8), (6, 384, 8), (5, 1000, 33),
                                   (3, 1024, 64)])
def test_sizes(T, E, k, score, dtype):
    rng = np.random.default_rng([T, E, k, len(dtype)])
    z, zd = make_logits(rng, T, E, dtype)
    bias = (rng.normal(size=E) * 0.1).astype(np.float32)
    for renormalise in (False, True):
        check_route(z, zd, score=score, top_k=k, renormalise=renormalise)
        check_route(z, zd, score=score, top_k=k, renormalise=renormalise, bias=bias, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,kept", [(5, 8, 2, 4, 2), (9, 6, 3, 3, 2), (40, 64, 6, 8, 3),
                                          (70, 256, 8, 8, 4), (7, 256, 4, 64, 5),
                                          (4, 1024, 16, 128, 20), (3, 30, 1, 30, 7),
                                          (8, 160, 6, 8, 3), (5, 1000, 9, 10, 1),
                                          (6, 512, 8, 4, 4), (3, 1024, 4, 1024, 9),
                                          (9, 12, 5, 2, 1), (5, 286, 10, 2, 2), (7, 160, 6, 8, 5),
                                          (4, 165, 3, 11, 6), (6, 34, 4, 17, 9), (3, 990, 8, 3, 2)])
def test_groups(T, E, k, G, kept, score):
    rng = np.random.default_rng([T, E, G])
    z, zd = make_logits(rng, T, E, "f32")
    bias = (rng.normal(size=E) * 0.1).astype(np.float32)
    for top in (1, 2):
        if E // G * kept < k:
            continue
        for b in (None, bias):
            check_route(z, zd, score=score, top_k=k, groups=G, kept_groups=kept, group_top=top,
                        bias=b, scale=2.5)


@pytest.mark.parametrize("E,G", [(8, 1), (64, 1), (256, 8), (100, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_and_near_ties(E, G, score):
    rng = np.random.default_rng(3)
    k = 5
    kept = max(1, G // 2)
    # all equal, two values, coarse steps, and values one float32 step apart
    z = np.zeros((24, E), np.float32)
    z[6:12] = rng.integers(0, 2, size=(6, E))
    z[12:18] = rng.integers(-4, 5, size=(6, E)) / 8
    near = np.float32(0.75) + np.arange(6).astype(np.float32) * np.float32(2.0 ** -24)
    z[18:] = rng.choice(near, size=(6, E))
    zt = torch.from_numpy(z)
    for bias in (None, np.zeros(E, np.float32),
                 (rng.integers(0, 2, size=E) / 1024).astype(np.float32)):
        check_route(zt, z, score=score, top_k=k, groups=G, kept_groups=kept, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("E", [16, 100, 512])
def test_masked_and_infinite(E, G, score):
    rng = np.random.default_rng(11)
    z = rng.normal(size=(12, E)).astype(np.float32)
    z[0] = -np.inf
    z[1] = np.nan
    z[2] = -np.inf
    z[2, E - 1] = 1.0
    z[3, ::2] = -np.inf
    z[4, ::3] = np.nan
    z[5, 3] = np.inf
    z[6, 2:9] = np.inf
    z[7] = np.finfo(np.float32).min
    z[8, 1:] = np.finfo(np.float32).min
    z[9, : E // 2] = -np.inf
    z[10] = -300.0
    z[10, 5] = 80.0
    bias = rng.normal(size=E).astype(np.float32)
    bias[1] = -np.inf
    bias[2] = np.nan
    live = np.ones(12, np.uint8)
    live[11] = 0
    for renormalise in (False, True):
        for b in (None, bias):
            check_route(torch.from_numpy(z), z, score=score, top_k=4, groups=G,
                        kept_groups=max(1, G // 2), bias=b, renormalise=renormalise, live=live)
    check_route(torch.from_numpy(z), z, score=score, top_k=4, live=live.astype(bool))


def test_strided_rows_and_offsets():
    rng = np.random.default_rng(2)
    dev = device()
    for dtype in DTYPES.values():
        wide = torch.from_numpy(rng.normal(size=(20, 150))).to(dtype).to(dev)
        for view in (wide[:, 1:129], wide[::2, 22:150], wide[3:4, :128], wide[:, 5:70]):
            check_route(view, view.double().cpu().numpy(), top_k=6)
            ids, _ = lib().route_experts(view, 6, renormalise=False)
            grad = torch.ones(view.shape[0], 6, device=dev)
            out = torch.full((view.shape[0], 200), 7.0, dtype=dtype, device=dev)
            lib().route_experts_backward(view, ids, grad, renormalise=False,
                                         out=out[:, 3:3 + view.shape[1]])
            assert bool((out[:, :3] == 7).all())
            assert bool((out[:, 3 + view.shape[1]:] == 7).all())
            again = lib().route_experts_backward(view.contiguous(), ids, grad, renormalise=False)
            assert torch.equal(again, out[:, 3:3 + view.shape[1]])


def test_no_tokens():
    dev = device()
    z = torch.zeros(0, 16, device=dev)
    ids, w, counts = lib().route_experts(z, 4, counts=True)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert counts.tolist() == [0] * 16
    assert lib().route_experts_backward(z, ids, w).shape == (0, 16)


def test_rows_more_than_2_to_31_elements_apart():
    rng = np.random.default_rng(15)
    stride = 2 ** 31 + 24
    flat = torch.empty(2 * stride + 64, dtype=torch.bfloat16, device=device())
    apart = flat.as_strided((3, 64), (stride, 1))
    z, zd = make_logits(rng, 3, 64, "bf16")
    apart.copy_(z)
    check_route(apart, zd, top_k=6, score="sigmoid")
    ids, w = lib().route_experts(apart, 6)
    want = lib().route_experts_backward(z.to(device()), ids, w)
    assert lib().route_experts_backward(apart, ids, w, out=apart) is apart
    assert torch.equal(apart, want)


def test_many_tokens():
    rng = np.random.default_rng(8)
    z, zd = make_logits(rng, 3001, 72, "bf16")
    bias = (rng.normal(size=72) * 0.05).astype(np.float32)
    check_route(z, zd, top_k=6, score="sigmoid", bias=bias, groups=8, kept_groups=3, scale=2.5)


# ------------------------------------------------------------------ gradient

def check_back(z, zd, ids, g, score, renormalise, scale):
    note("route_back %s k=%d %s %s" % (tuple(z.shape), ids.shape[1], score, renormalise))
    dev = device()
    got = lib().route_experts_backward(z.to(dev), torch.from_numpy(ids).to(dev),
                                       torch.from_numpy(g).to(dev), score, renormalise, scale)
    assert got.dtype == z.dtype
    want, size = plain.route_backward(zd, ids, g, score, renormalise, scale)
    there = zd > -np.inf
    low = np.where(there, zd, np.inf).min(axis=1, keepdims=True)
    high = np.where(there, zd, -np.inf).max(axis=1, keepdims=True)
    L = np.where(np.isfinite(high - low), high - low, 0.0)
    tol = (2 * L + 70 + ids.shape[1]) * 2.0 ** -24 * size
    tol = tol + np.abs(want) * torch.finfo(z.dtype).eps / 2
    tol = tol + float(torch.finfo(z.dtype).tiny)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 7, 7), (65, 60, 4), (33, 64, 6),
                                   (9, 130, 8), (40, 256, 8), (5, 1000, 33), (3, 1024, 64)])
def test_gradient(T, E, k, renormalise, score, dtype):
    rng = np.random.default_rng([T, E, k])
    z, zd = make_logits(rng, T, E, dtype)
    ids, _, _ = plain.route(zd, k, score)
    g = rng.normal(size=(T, k)).astype(np.float32)
    check_back(z, zd, ids, g, score, renormalise, 1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_gradient_of_empty_and_masked_places(renormalise, score):
    rng = np.random.default_rng(4)
    z = rng.normal(size=(8, 20)).astype(np.float32)
    z[0, 3:] = -np.inf
    z[1] = -np.inf
    z[2, 5] = np.nan
    ids, _, _ = plain.route(z, 5, score, live=[1, 1, 1, 0, 1, 1, 1, 1])
    assert (ids[1] == -1).all() and (ids[3] == -1).all() and (ids[0, 3:] == -1).all()
    ids[4] = [2, -1, 7, 20, -9]
    g = rng.normal(size=(8, 5)).astype(np.float32)
    g[ids < 0] = np.nan   # nothing of an empty place may get through
    check_back(torch.from_numpy(z), z.astype(np.float64), ids, g, score, renormalise, 2.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("E", [20, 600])
def test_gradient_of_infinite_logits(E, renormalise, score):
    rng = np.random.default_rng(E + 1)
    z = rng.normal(size=(6, E)).astype(np.float32)
    z[0, 3] = np.inf
    z[1, [2, 11]] = np.inf
    z[2, 5:] = np.finfo(np.float32).min
    z[3] = np.finfo(np.float32).min
    z[4, 7] = np.finfo(np.float32).max
    ids, _, _ = plain.route(z.astype(np.float64), 4, score)
    g = rng.normal(size=(6, 4)).astype(np.float32)
    check_back(torch.from_numpy(z), z.astype(np.float64), ids, g, score, renormalise, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("offset", [-90.0, -200.0, -600.0, 90.0])
def test_gradient_of_far_logits(offset, renormalise, score, dtype):
    """Scores that float32 does not hold, shares of their sum that it does."""
    rng = np.random.default_rng(int(abs(offset)))
    z, zd = make_logits(rng, 8, 40, dtype)
    z = (z.float() + offset).to(z.dtype)
    zd = z.double().numpy()
    ids, _, _ = plain.route(zd, 6, score)
    g = rng.normal(size=(8, 6)).astype(np.float32)
    check_back(z, zd, ids, g, score, renormalise, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("E", [9, 200, 700])
def test_gradient_of_an_index_that_comes_twice(E, renormalise, score):
    """w_i = s[id_i] / sum over the places: every place adds its term."""
    rng = np.random.default_rng(E)
    z = rng.normal(size=(6, E)).astype(np.float32)
    ids = rng.integers(0, 4, size=(6, 20)).astype(np.int32)
    ids[0] = 3
    g = rng.normal(size=(6, 20)).astype(np.float32)
    check_back(torch.from_numpy(z), z.astype(np.float64), ids, g, score, renormalise, 1.0)
    dev = device()
    on = [torch.from_numpy(a).to(dev) for a in (z, ids, g)]
    first = lib().route_experts_backward(*on, score, renormalise)
    for _ in range(5):
        assert torch.equal(first, lib().route_experts_backward(*on, score, renormalise))


def test_gradient_against_differences_of_the_forward():
    """The library's own forward, in float32: a step of 2^-6 moves a weight
    by at most 2^-6, its float32 value is off by 2^-21 of at most 1, and the
    third derivative of a weight is below 1, so that a difference quotient is
    off by 2 * 2^-21 / 2^-5 + 2^-12 / 6 < 2^-12, times the sum of |g|."""
    rng = np.random.default_rng(6)
    dev = device()
    T, E, k, h = 4, 12, 3, 2.0 ** -6
    # far enough apart that a step changes no choice
    base = np.stack([rng.permutation(E) for _ in range(T)]).astype(np.float32) / 4
    for score in ("softmax", "sigmoid"):
        for renormalise in (False, True):
            z = torch.from_numpy(base).to(dev)
            ids, _ = lib().route_experts(z, k, score=score, renormalise=renormalise)
            g = torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32)).to(dev)
            grad = lib().route_experts_backward(z, ids, g, score, renormalise).cpu().numpy()
            bound = 2.0 ** -12 * g.abs().sum(dim=1).cpu().numpy()
            for j in range(E):
                sides = []
                for sign in (1, -1):
                    y = z.clone()
                    y[:, j] += sign * h
                    i2, w = lib().route_experts(y, k, score=score, renormalise=renormalise)
                    assert torch.equal(i2, ids)
                    sides.append((w.double() * g.double()).sum(dim=1).cpu().numpy())
                assert np.all(np.abs((sides[0] - sides[1]) / (2 * h) - grad[:, j]) <= bound)


# ------------------------------------------------- streams, graphs, refusals

def test_other_stream_and_graph_replays():
    dev = device()
    rng = np.random.default_rng(9)
    z = torch.empty(50, 96, device=dev)
    g = torch.from_numpy(rng.normal(size=(50, 4)).astype(np.float32)).to(dev)
    side = torch.cuda.Stream()
    inputs = [torch.from_numpy(rng.normal(size=(50, 96)).astype(np.float32)).to(dev)
              for _ in range(4)]
    z.copy_(inputs[0])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib().route_experts(z, 4, counts=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, w, counts = lib().route_experts(z, 4, counts=True)
        grad = lib().route_experts_backward(z, ids, g)
    for x in inputs:
        z.copy_(x)
        graph.replay()
        eager = lib().route_experts(x, 4, counts=True)
        for a, b in zip((ids, w, counts), eager):
            assert torch.equal(a, b)
        assert torch.equal(grad, lib().route_experts_backward(x, eager[0], g))
        torch.cuda.synchronize()


def test_refusals():
    dev = device()
    g = lib()
    z = torch.zeros(4, 8, device=dev)
    for kw in (dict(top_k=0), dict(top_k=9), dict(top_k=2, groups=3),
               dict(top_k=2, scale=math.nan), dict(top_k=2, group_top=3),
               dict(top_k=3, groups=4, kept_groups=1), dict(top_k=2, groups=0),
               dict(top_k=-1)):
        with pytest.raises(g.NMSError) as e:
            g.route_experts(z, **kw)
        assert e.value.status == "NMS_INVALID_ARG"
    with pytest.raises(g.NMSError) as e:
        g.route_experts(torch.zeros(2, 1025, device=dev), 2)
    assert e.value.status == "NMS_TOO_LARGE"
    with pytest.raises(ValueError):
        g.route_experts(z, 2, score="relu")
    for kw in (dict(top_k=2 ** 32 + 2), dict(top_k=2, groups=2 ** 32 + 1),
               dict(top_k=2, kept_groups=2 ** 32 + 1), dict(top_k=2, group_top=2 ** 32 + 1)):
        with pytest.raises(ValueError):
            g.route_experts(z, **kw)
    with pytest.raises(TypeError):
        g.route_experts(z, 2.5)
    with pytest.raises(TypeError):
        g.route_experts(z, 2, live=[1, 1, 1, 1])
    with pytest.raises(TypeError):
        g.route_experts(z.double(), 2)
    with pytest.raises(ValueError):
        g.route_experts(z.t(), 2)
    with pytest.raises(ValueError):
        g.route_experts(z, 2, bias=torch.zeros(7, device=dev))
    with pytest.raises(ValueError):
        g.route_experts(z, 2, bias=torch.zeros(8))
    with pytest.raises(TypeError):
        g.route_experts(z, 2, live=torch.zeros(4, device=dev))
    ids, w = g.route_experts(z, 2)
    with pytest.raises(ValueError):
        g.route_experts_backward(z, ids[:3], w)
    with pytest.raises(TypeError):
        g.route_experts_backward(z, ids.long(), w)
    with pytest.raises(TypeError):
        g.route_experts_backward(z, ids, w.half())
    with pytest.raises(TypeError):
        g.route_experts_backward(z, ids, w, out=torch.empty(4, 8, dtype=torch.half, device=dev))
    with pytest.raises(ValueError):
        g.route_experts_backward(z, ids, w, out=torch.empty(4, 9, device=dev))
