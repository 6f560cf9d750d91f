"""The losses as they are used: after routing and picking, through autograd, on
other streams, in graphs, in place, at sizes that are streamed."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gpu_util import device, note  # noqa: E402
from loss_util import TYPES, U, Bounds, dev, host, lib, logits_of, within  # noqa: E402
from oracle import losses as plain  # noqa: E402
from test_gpu_losses import policy_inputs, tokens_of  # noqa: E402

pytestmark = pytest.mark.gpu


def normal(rng, *shape):
    return torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(device())


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", TYPES)
def test_picked_and_trained(dtype):
    """Tokens picked at several temperatures, scored, and trained on: the log
    probabilities of both calls agree, so that the first ratio is 1 and the
    policy loss is minus the mean advantage; the gradients agree with those of the
    log probabilities."""
    note("picked and trained %s" % dtype)
    rng = np.random.default_rng(0)
    g = lib()
    T, V = 40, 5003
    z = logits_of(rng, T, V, dtype)
    z[:, 3::7] = -float("inf")
    heat = (0.4 + rng.random(T)).astype(np.float32)
    heat[::8] = 0.0
    ids, lp = g.pick_tokens(z, dev(rng.random(T).astype(np.float32)), max_top_k=200,
                            temperature=dev(heat))
    b = Bounds(host(z), ids.cpu().numpy(), heat)
    got = g.token_logprobs(z, ids, temperature=dev(heat))
    within(host(got), b.lp, b.logprob, "logprobs")
    # (pick_tokens states 7e-6 and its rounding)
    assert np.all(np.abs(host(lp) - b.lp) <= 7e-6 + U * np.abs(b.lp))
    adv = dev(rng.normal(size=T).astype(np.float32))
    loss, dz, again = g.policy_loss_with_grad(z, ids, got, adv, temperature=dev(heat))
    assert torch.equal(again, got)
    # each ratio is exp of a difference of 2^-25 of the log probability at most
    err = (np.abs(host(adv)) * (U * np.abs(b.lp) + 6 * U)).mean()
    assert abs(float(loss) + float(adv.double().mean())) <= err + U * abs(float(loss))
    by = g.token_logprobs_backward(z, ids, -adv / T, temperature=dev(heat))
    want = plain.combine(b.counts, b.dlp, b.dh, -host(adv) / T, None)
    tol = b.grad(dtype, want, host(adv) / T, None, np.abs(host(adv)) / T * (U * np.abs(b.lp) + 6 * U))
    within(host(by), want, tol, "gradient of log probabilities")
    within(host(dz), want, tol, "gradient of the policy loss")


def test_a_step_of_a_model_with_experts():
    """Experts by route_experts, their balance, and a policy loss behind them: one
    backward pass, its gradients against differences in 64 bits."""
    note("a step with experts")
    rng = np.random.default_rng(1)
    g = lib()
    T, D, E, V, k = 24, 6, 8, 30, 2
    x = normal(rng, T, D)
    router, experts, head = normal(rng, D, E), normal(rng, E, D) * 0.5, normal(rng, D, V)
    tokens = dev(rng.integers(0, V, T).astype(np.int32))
    old, adv = dev(np.full(T, -3.0, np.float32)), dev(rng.normal(size=T).astype(np.float32))

    def step(router, experts, head):
        logits = (x[:, :, None] * router[None]).sum(1)
        ids, w = g.route_experts(logits, k)
        balance, _ = g.balance_loss(logits, ids, balance=0.1, z=0.01)
        mixed = (w[:, :, None] * experts[ids.long()]).sum(1)
        out = ((x + mixed)[:, :, None] * head[None]).sum(1)
        policy, _ = g.policy_loss(out, tokens, old, adv, clip=0.9, clip_high=5.0)
        return policy + balance, ids

    params = [p.clone().requires_grad_() for p in (router, experts, head)]
    loss, ids = step(*params)
    loss.backward()
    ids_np, adv_np, tok = ids.cpu().numpy(), host(adv), tokens.cpu().numpy()

    def exact(router, experts, head):
        xd = host(x)
        logits = xd @ router
        chosen = np.take_along_axis(logits, ids_np, 1)
        w = np.exp(chosen - chosen.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        mixed = (w[:, :, None] * experts[ids_np]).sum(1)
        policy = plain.policy((xd + mixed) @ head, tok, np.full(T, -3.0), adv_np, clip=0.9,
                              clip_high=5.0)[0]
        return policy + plain.balance(logits, ids_np, balance=0.1, z=0.01)[0]

    values = [host(p) for p in (router, experts, head)]
    loss = float(loss.detach())
    assert abs(loss - exact(*values)) <= (T * D + V) * U * max(1.0, abs(loss))
    for i, p in enumerate(params):
        for at in [tuple(rng.integers(0, n) for n in p.shape) for _ in range(6)]:
            step_size, side = 1e-5, []
            for s in (1, -1):
                v = [a.copy() for a in values]
                v[i][at] += s * step_size
                side.append(exact(*v))
            want = (side[0] - side[1]) / (2 * step_size)
            # float32 products and sums of up to T * D + V terms, and the difference's 1e-10
            size = float(p.grad.abs().max())
            assert abs(float(p.grad[at]) - want) <= (T * D + V) * U * size + 1e-8, (i, at)


# ------------------------------------------------------------------ autograd

def test_gradients_of_log_probabilities_and_entropies():
    rng = np.random.default_rng(2)
    g = lib()
    z, a = normal(rng, 9, 300), dev(tokens_of(rng, 9, 300))
    f, h = normal(rng, 9), normal(rng, 9)

    def grad(use):
        leaf = z.clone().requires_grad_()
        lp, ent = g.token_logprobs(leaf, a, entropy=True)
        assert lp.requires_grad and ent.requires_grad
        use(lp, ent).backward()
        return leaf.grad

    back = lambda p, e: g.token_logprobs_backward(z, a, p, None, e)  # noqa: E731
    zero, ones = torch.zeros_like(f), torch.ones_like(f)
    assert torch.equal(grad(lambda lp, ent: (lp * f + ent * h).sum()), back(f, h))
    assert torch.equal(grad(lambda lp, ent: (lp * f).sum()), back(f, None))
    assert torch.equal(grad(lambda lp, ent: (ent * h).sum()), back(zero, h))
    assert torch.equal(grad(lambda lp, ent: ent.sum() + lp.sum()), back(ones, ones))
    # strided upstream, strided logits
    wide = normal(rng, 9, 700)
    leaf = wide[:, 5:305].detach().requires_grad_()
    lp = g.token_logprobs(leaf, a)
    lp[::2].sum().backward()
    mask = zero.clone()
    mask[::2] = 1
    assert torch.equal(leaf.grad, g.token_logprobs_backward(leaf.detach(), a, mask))


def test_losses_keep_their_inputs_and_have_no_second_gradient():
    rng = np.random.default_rng(3)
    g = lib()
    z, tokens, old, adv, w, ref = policy_inputs(rng, 12, 90, torch.float32)
    a, old, adv, w, ref = (dev(v) for v in (tokens, old, adv, w, ref))
    at = dev(np.array([0, 3, 6, 9, 12]))
    ids = dev(rng.integers(0, 90, (12, 2)).astype(np.int32))
    calls = [lambda x: g.policy_loss(x, a, old, adv, w, ref, kl=0.1, entropy=0.01)[0],
             lambda x: g.preference_loss(x, a, at)[0],
             lambda x: g.balance_loss(x, ids, z=0.1)[0],
             lambda x: g.token_logprobs(x, a).sum()]
    for call in calls:
        # twice through the same graph
        leaf = z.clone().requires_grad_()
        loss = call(leaf)
        loss.backward(retain_graph=True)
        first = leaf.grad.clone()
        loss.backward()
        assert torch.equal(leaf.grad, first * 2) and bool((first != 0).any())
        # logits that change before the backward pass
        leaf = z.clone().requires_grad_()
        y = leaf * 1.0
        loss = call(y)
        y.add_(1.0)
        with pytest.raises(RuntimeError):
            loss.backward()
        # a gradient of the gradient
        leaf = z.clone().requires_grad_()
        (grad,) = torch.autograd.grad(call(leaf), leaf, create_graph=True)
        with pytest.raises(RuntimeError):
            grad.sum().backward()
        # no graph where none is wanted
        with torch.no_grad():
            assert not call(leaf).requires_grad
        assert not call(z).requires_grad
    adv2 = adv.clone()
    leaf = z.clone().requires_grad_()
    loss = g.policy_loss(leaf, a, old, adv2)[0]
    adv2.zero_()
    with pytest.raises(RuntimeError):
        loss.backward()


def test_what_out_overwrites():
    rng = np.random.default_rng(4)
    g = lib()
    z, tokens, old, adv, w, _ = policy_inputs(rng, 12, 90, torch.float32)
    a, old, adv, w = (dev(v) for v in (tokens, old, adv, w))
    at = dev(np.array([0, 5, 12]))
    ids = dev(rng.integers(0, 90, (12, 2)).astype(np.int32))
    calls = [lambda x, out: g.policy_loss_with_grad(x, a, old, adv, w, out=out)[1],
             lambda x, out: g.preference_loss_with_grad(x, a, at, out=out)[1],
             lambda x, out: g.balance_loss_with_grad(x, ids, out=out)[1],
             lambda x, out: g.token_logprobs_backward(x, a, adv, out=out)]
    for call in calls:
        want = call(z, None)
        out = torch.empty_like(z)
        version = out._version
        assert call(z, out) is out and out._version > version and torch.equal(out, want)
        there = z.clone()
        assert call(there, there) is there and torch.equal(there, want)
        with pytest.raises(RuntimeError):
            call(z, torch.empty_like(z).requires_grad_())
        for bad in (torch.empty(12, 91, device=device()), torch.empty(12, 90),
                    torch.empty(90, 12, device=device()).t()):
            with pytest.raises(ValueError):
                call(z, bad)
        with pytest.raises(TypeError):
            call(z, torch.empty(12, 90, device=device(), dtype=torch.float16))
        y = (z.clone().requires_grad_()).exp()      # its gradient needs y
        with torch.no_grad():
            call(y, y)
        with pytest.raises(RuntimeError):
            y.sum().backward()
        with torch.inference_mode():                # no versions there
            x = torch.ones(12, 90, device=device())
            call(x, x)


def test_the_gradient_that_a_call_returns_goes_on():
    """torch.autograd.backward takes it from there."""
    rng = np.random.default_rng(5)
    g = lib()
    x, head = normal(rng, 10, 4), normal(rng, 4, 50).requires_grad_()
    z, a = (x[:, :, None] * head[None]).sum(1), dev(tokens_of(rng, 10, 50, 0.0))
    old, adv = normal(rng, 10), normal(rng, 10)
    _, dz, _ = g.policy_loss_with_grad(z, a, old, adv)
    torch.autograd.backward(z, dz)
    first = head.grad.clone()
    head.grad = None
    g.policy_loss((x[:, :, None] * head[None]).sum(1), a, old, adv)[0].backward()
    assert torch.equal(head.grad, first)


# ---------------------------------------------------------- streams and graphs

def all_calls(g, z, a, old, adv, w, ref, at, router, ids, live, offsets, up):
    """Every entry point on the same inputs, as a list of tensors."""
    out = list(g.token_logprobs(z, a, entropy=True))
    out.append(g.token_logprobs_backward(z, a, adv, grad_entropies=old))
    out += g.policy_loss_with_grad(z, a, old, adv, w, ref, kl=0.1, entropy=0.01, grad_loss=up)
    out += g.policy_loss(z, a, old, adv)
    out += g.preference_loss_with_grad(z, a, at, grad_loss=up)
    out += g.preference_loss(z, a, at, kind="hinge", average=True)
    out += g.balance_loss_with_grad(router, ids, "sigmoid", z=0.1, live=live, offsets=offsets,
                                    grad_loss=up)
    out += g.balance_loss(router, ids, live=live)
    return out


def inputs(rng, T, V, dtype=torch.float32, E=20):
    z, tokens, old, adv, w, ref = policy_inputs(rng, T, V, dtype)
    at = np.sort(rng.integers(0, T + 1, 7)).astype(np.int64)
    ids = rng.integers(-1, E, (T, 3)).astype(np.int32)
    offsets = np.array([0, T // 3, T], np.int64)
    up = np.float32([rng.random() + 0.5])
    return [z] + [dev(v) for v in (tokens, old, adv, w, ref, at)] + [
        logits_of(rng, T, E, dtype), dev(ids), dev(rng.random(T) < 0.8), dev(offsets), dev(up)]


@pytest.mark.parametrize("T,V", [(6, 70), (9, 70001), (70, 33000), (1100, 40)])
def test_the_same_bits_every_time(T, V):
    """Also on another stream and after other calls on the same workspace."""
    note("the same bits %d %d" % (T, V))
    rng = np.random.default_rng(6)
    g = lib()
    given = inputs(rng, T, V)
    want = [t.clone() for t in all_calls(g, *given)]
    all_calls(g, *inputs(rng, 13, 900))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = all_calls(g, *given)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b, c in zip(want, all_calls(g, *given), there):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("T,V", [(6, 70), (9, 70001), (70, 33000)])
def test_captured_calls(T, V):
    """Replays with new contents, eager work and synchronisation between them."""
    note("captured %d %d" % (T, V))
    rng = np.random.default_rng(7)
    g = lib()
    sets = [inputs(rng, T, V) for _ in range(4)]
    static = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        all_calls(g, *static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_calls(g, *static)
    for given in sets + sets[:2]:
        for s, t in zip(static, given):
            s.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, all_calls(g, *given)):
            assert torch.equal(a, b)


def test_two_graphs_at_the_same_time():
    """Each has a workspace of its own."""
    note("two graphs")
    rng = np.random.default_rng(8)
    g = lib()
    sets = [inputs(rng, 80, 40001) for _ in range(2)]
    want = [[t.clone() for t in all_calls(g, *given)] for given in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for given in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(all_calls(g, *given))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for stream, graph in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            for s, t in zip(a, b):
                assert torch.equal(s, t)


def test_a_step_captured_with_its_backward_pass():
    note("captured step")
    rng = np.random.default_rng(9)
    g = lib()
    sets = [inputs(rng, 30, 200) for _ in range(3)]
    static = [t.clone() for t in sets[0]]
    leaves = [static[0].requires_grad_(), static[7].requires_grad_()]

    def step(z, a, old, adv, w, ref, at, router, ids, live, offsets, up):
        ids, gates = g.route_experts(router, 3, live=live)
        lp, h = g.token_logprobs(z, a, entropy=True)
        loss = (g.policy_loss(z, a, old, adv, w)[0] + g.preference_loss(z, a, at)[0] +
                g.balance_loss(router, ids, z=0.1, live=live)[0] + (gates * gates).sum() +
                (lp * adv).sum() + h.sum())
        return torch.autograd.grad(loss, [z, router])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            first = step(*static)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    del first
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*static)
    got = []
    for given in sets + sets[:1]:
        with torch.no_grad():
            for s, t in zip(static, given):
                s.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        got.append([t.clone() for t in out])
    del graph, out, leaves
    for given, have in zip(sets + sets[:1], got):
        fresh = [t.clone() for t in given]
        fresh[0].requires_grad_()
        fresh[7].requires_grad_()
        for a, b in zip(have, step(*fresh)):
            assert torch.equal(a, b)


# ------------------------------------------------------------- sizes that stream

@pytest.mark.parametrize("T,V,dtype", [(1500, 65537, torch.bfloat16), (700, 131080, torch.float16),
                                       (320, 140001, torch.float32), (21000, 4100, torch.bfloat16),
                                       (5000, 17003, torch.float16)])
def test_sizes_past_the_caches(T, V, dtype):
    """Gradients of more than 160 MB: a few rows against the plain form, all of
    them finite, and in place the same."""
    note("past the caches %d %d %s" % (T, V, dtype))
    rng = np.random.default_rng(10)
    g = lib()
    seeded = torch.Generator(device=device())
    seeded.manual_seed(T)
    z = torch.randn(T, V, generator=seeded, device=device()).mul_(2.5).to(dtype)
    tokens = tokens_of(rng, T, V)
    w = (rng.random(T) * (rng.random(T) < 0.8)).astype(np.float32)
    # (ratios near 1: 64 w A times one of 10^4 is past float16)
    old = (host(g.token_logprobs(z, dev(tokens))) + 0.4 * rng.normal(size=T)).astype(np.float32)
    adv = rng.normal(size=T).astype(np.float32)
    at = np.array([0, T // 4, T // 2, 3 * T // 4, T - 3], np.int64)
    rows = np.array([0, 1, T // 2, T - 2, T - 1] + rng.integers(0, T, 5).tolist())
    sample = host(z[torch.from_numpy(rows).to(z.device)])
    given = [dev(v) for v in (tokens, old, adv, w)]
    up = dev(np.float32([64.0]))
    loss, dz, lp = g.policy_loss_with_grad(z, *given, grad_loss=up)
    b = Bounds(sample, tokens[rows], None, w[rows])
    within(host(lp)[rows], b.lp, b.logprob, "logprobs")
    ratio = np.exp(b.lp - old[rows])
    free, held = ratio * adv[rows], np.clip(ratio, 0.8, 1.2) * adv[rows]
    c = np.where(b.counts, -64.0 * w[rows] * np.where(free <= held, free, 0.0), 0.0)
    want = plain.combine(b.counts, b.dlp, b.dh, c, None)
    dg = np.abs(64.0 * w[rows] * free) * (b.logprob + 7 * U)
    within(host(dz[torch.from_numpy(rows).to(z.device)]), want, b.grad(dtype, want, c, None, dg),
           "policy")
    assert bool(torch.isfinite(dz).all())
    one, dp, sums, margins = g.preference_loss_with_grad(z, given[0], dev(at), beta=0.001,
                                                         average=True, grad_loss=up)
    b = Bounds(sample, tokens[rows])
    # 64 * slope * beta / rows that count, of each sequence
    counts = (tokens >= 0) & (tokens < V)
    h = host(margins)
    slope = -1.0 / (1.0 + np.exp(h)) / 2
    c = np.zeros(T)
    for q in range(4):
        own = slice(at[q], at[q + 1])
        c[own] = 64.0 * slope[q % 2] * 0.001 / counts[own].sum() * (1 if q < 2 else -1)
    c = np.where(b.counts, c[rows], 0.0)
    want = plain.combine(b.counts, b.dlp, b.dh, c, None)
    within(host(dp[torch.from_numpy(rows).to(z.device)]), want,
           b.grad(dtype, want, c, None, 8 * U * np.abs(c)), "preference")
    assert bool((dp[T - 3:] == 0).all())
    back = g.token_logprobs_backward(z, given[0], given[2])
    c = adv[rows].astype(np.float64)
    want = plain.combine(b.counts, b.dlp, b.dh, c, None)
    within(host(back[torch.from_numpy(rows).to(z.device)]), want, b.grad(dtype, want, c), "backward")
    g.policy_loss_with_grad(z, *given, grad_loss=up, out=z)
    assert torch.equal(z, dz)
