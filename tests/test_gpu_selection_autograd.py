"""The selection operators on tensors that require a gradient."""
import numpy as np
import pytest

from gpu_util import device, note
from oracle import selection as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

OPTIONS = [dict(score="softmax", renormalise=False), dict(score="softmax", renormalise=True),
           dict(score="sigmoid", renormalise=False, scale=2.5),
           dict(score="sigmoid", renormalise=True, scale=2.5, groups=4, kept_groups=2)]


def lib():
    import greedy_iou_nms_amd as g
    return g


def normal(rng, *shape):
    return torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(device())


# ------------------------------------------------------------------- routing

@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("options", OPTIONS)
def test_weights_carry_their_gradient(options, dtype):
    """The gradient that autograd gets is the explicit call's, bit for bit."""
    note("autograd %s %s" % (options, dtype))
    rng = np.random.default_rng(1)
    g = lib()
    z = normal(rng, 37, 48).to(dtype).requires_grad_()
    factor = normal(rng, 37, 5)
    bias = normal(rng, 48) * 0.1
    live = torch.from_numpy(rng.random(37) < 0.8).to(device())
    ids, w, counts = g.route_experts(z, 5, bias=bias, live=live, counts=True, **options)
    assert w.requires_grad and not ids.requires_grad and not counts.requires_grad
    with torch.no_grad():
        eager = g.route_experts(z, 5, bias=bias, live=live, counts=True, **options)
    assert not any(t.requires_grad for t in eager)
    for a, b in zip((ids, w, counts), eager):
        assert torch.equal(a, b)
    (w * factor).sum().backward()
    back = {k: v for k, v in options.items() if k in ("score", "renormalise", "scale")}
    want = g.route_experts_backward(z.detach(), ids, factor, **back)
    assert z.grad.dtype == dtype and torch.equal(z.grad, want)
    assert bool((z.grad[~live] == 0).all()) and bool((z.grad != 0).any())


def test_a_router_learns_through_the_call():
    """Gradients of the layers before the call, against the formula's: the
    router's weights x^T dz, whose dz is the plain one in 64 bits.  dz is off by
    (2 L + 70 + k) 2^-24 of its terms' absolute sum (see test_gpu_route.py, L the
    largest distance of a row's logits), a sum of T products adds T 2^-24."""
    rng = np.random.default_rng(2)
    T, D, E, k = 64, 16, 24, 4
    x, router = normal(rng, T, D), (normal(rng, D, E) * 0.3).requires_grad_()
    factor = normal(rng, T, k)
    logits = (x[:, :, None] * router[None]).sum(1)
    ids, w = lib().route_experts(logits, k, score="sigmoid", scale=2.0)
    (w * factor).sum().backward()
    zd = logits.detach().double().cpu().numpy()
    dz, size = plain.route_backward(zd, ids.cpu().numpy(), factor.cpu().numpy(), "sigmoid", True,
                                    2.0)
    xd = x.double().cpu().numpy()
    L = float((zd.max(axis=1) - zd.min(axis=1)).max())
    tol = (2 * L + 70 + k + T + 2) * 2.0 ** -24 * (np.abs(xd).T @ size)
    err = np.abs(router.grad.double().cpu().numpy() - xd.T @ dz)
    assert np.all(err <= tol + np.finfo(np.float32).tiny)


def test_expanded_strided_and_unused_gradients():
    rng = np.random.default_rng(3)
    g = lib()
    wide = normal(rng, 20, 90)
    z = wide[::2, 5:69].detach().requires_grad_()
    assert not z.is_contiguous()
    ids, w = g.route_experts(z, 6, renormalise=False)
    w.sum().backward()          # an expanded gradient
    ones = torch.ones(10, 6, device=z.device)
    assert torch.equal(z.grad, g.route_experts_backward(z.detach(), ids, ones, renormalise=False))
    z.grad = None
    ids, w = g.route_experts(z, 6, renormalise=False)
    w.t()[1].sum().backward()   # of one column, through a transposed view
    ones[:, 0] = 0
    ones[:, 2:] = 0
    assert torch.equal(z.grad, g.route_experts_backward(z.detach(), ids, ones, renormalise=False))
    # a scale that has changed by the time of the backward pass
    scale = torch.tensor(3.0)
    z.grad = None
    ids, w = g.route_experts(z, 6, scale=scale)
    scale.fill_(100.0)
    factor = normal(rng, 10, 6)
    (w * factor).sum().backward()
    assert torch.equal(z.grad, g.route_experts_backward(z.detach(), ids, factor, scale=3.0))


def test_no_tokens_and_changed_logits():
    g = lib()
    z = torch.zeros(0, 16, device=device(), requires_grad=True)
    ids, w = g.route_experts(z, 4)
    w.sum().backward()
    assert z.grad.shape == (0, 16)
    x = torch.randn(4, 16, device=device(), requires_grad=True)
    y = x * 1.0
    ids, w = g.route_experts(y, 4)
    y.add_(1.0)                 # the backward pass needs them as they were
    with pytest.raises(RuntimeError):
        w.sum().backward()


def test_another_stream_and_a_captured_step():
    """On another stream, and captured with its backward pass: warmed up on a
    side stream, no eager graph of the same tensors alive while capturing."""
    rng = np.random.default_rng(4)
    g = lib()
    inputs = [normal(rng, 30, 40) for _ in range(4)]
    factor = normal(rng, 30, 3)

    def step(z):
        ids, w = g.route_experts(z, 3, score="sigmoid")
        return torch.autograd.grad((w * factor).sum(), z)[0]

    def explicit(x):
        ids, _ = g.route_experts(x, 3, score="sigmoid")
        return g.route_experts_backward(x, ids, factor, score="sigmoid")

    static = inputs[0].clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            first = step(static)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(first, explicit(inputs[0]))
    del first
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(static)
    for x in inputs:
        with torch.no_grad():
            static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, explicit(x))


# ------------------------------------------------- logits and tokens

def rules_and_logits(rng, B=3, V=500):
    g = lib()
    z = normal(rng, B, V).requires_grad_()
    history = torch.from_numpy(rng.integers(0, V, size=(B, 20)).astype(np.int32)).to(device())
    rules = g.LogitRules(V, history=history,
                         history_len=torch.full((B,), 20, dtype=torch.int32, device=device()),
                         repetition=torch.full((B,), 1.5, device=device()))
    return g, z, rules


def test_adjusted_logits_do_not_lose_a_gradient_silently():
    g, z, rules = rules_and_logits(np.random.default_rng(5))
    with torch.no_grad():
        want = g.adjust_logits(z, rules)
    assert not want.requires_grad
    out = g.adjust_logits(z, rules)
    assert out.requires_grad and torch.equal(out, want)
    with pytest.raises(NotImplementedError):
        (out.sum() + z.sum()).backward()
    assert not g.adjust_logits(z.detach(), rules).requires_grad
    for kw in (dict(logits=z, out=torch.empty_like(want)), dict(logits=z, out=z),
               dict(logits=want, out=torch.empty_like(want).requires_grad_())):
        before = z.detach().clone()
        with pytest.raises(RuntimeError):
            g.adjust_logits(kw["logits"], rules, out=kw["out"])
        assert torch.equal(z, before)
        with torch.no_grad():
            assert torch.equal(g.adjust_logits(kw["logits"].clone(), rules, out=kw["out"].clone()),
                               want if kw["logits"] is z else g.adjust_logits(want, rules))


def test_picked_tokens_do_not_lose_a_gradient_silently():
    g, z, rules = rules_and_logits(np.random.default_rng(6))
    u = torch.full((3,), 0.4, device=device())
    with torch.no_grad():
        want = g.pick_tokens(z, u, max_top_k=9, rules=rules)
    ids, lp = g.pick_tokens(z, u, max_top_k=9, rules=rules)
    assert torch.equal(ids, want[0]) and torch.equal(lp, want[1])
    assert not ids.requires_grad and lp.requires_grad and not want[1].requires_grad
    with pytest.raises(NotImplementedError):
        lp.sum().backward()


# ------------------------------------------------------- what out overwrites

def test_writing_to_out_is_seen_by_autograd():
    """A tensor that a backward pass needs, overwritten by a call in place: the
    pass must not go on with the new values."""
    g, z, rules = rules_and_logits(np.random.default_rng(7))
    y = z.exp()                                     # its gradient needs y
    with torch.no_grad():
        assert g.adjust_logits(y, rules, out=y) is y
    with pytest.raises(RuntimeError):
        y.sum().backward()
    other, x = torch.empty_like(z, requires_grad=False), normal(np.random.default_rng(8), 3, 500)
    g.adjust_logits(x, rules, out=other)
    version = other._version
    g.adjust_logits(x, rules, out=other)
    assert other._version > version
    ids, w = g.route_experts(x, 4)
    version = other._version
    assert g.route_experts_backward(x, ids, w, out=other) is other
    assert other._version > version
    with pytest.raises(RuntimeError):
        g.route_experts_backward(x, ids, w, out=torch.empty_like(x).requires_grad_())
    with torch.inference_mode():                    # no versions there
        x = torch.ones(3, 500, device=device())
        assert g.adjust_logits(x, rules, out=x) is x
        g.route_experts_backward(x, *g.route_experts(x, 4), out=x)
