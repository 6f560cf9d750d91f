"""Gradients of the losses where values are at the ends of their types: NaN and
infinities beside masked logits, temperatures whose inverse float32 does not
hold, against the plain 64-bit ones (bounds: loss_util.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gpu_util import note  # noqa: E402
from loss_util import TYPES, U, Bounds, dev, host, lib, logits_of, within  # noqa: E402
from oracle import losses as plain  # noqa: E402
from test_gpu_losses import policy_bounds, tokens_of  # noqa: E402

pytestmark = pytest.mark.gpu

# a row in a workgroup of 64 threads, of 1024, and shared by slices; of a workgroup
# that reads the end of its row again
SIZES = [(8, 9), (8, 300), (8, 9001), (8, 70001), (104, 70001)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("entropy", [False, True])
def test_gradients_of_rows_with_nan_and_infinity(T, V, dtype, entropy):
    """They are NaN throughout, also where a logit is masked or far below the
    others, and other rows' are not."""
    note("gradients of nan %d %d %s %s" % (T, V, dtype, entropy))
    rng = np.random.default_rng(V)
    z = logits_of(rng, T, V, dtype)
    z[:, 4::5] = -float("inf")
    z[:, 3] = torch.finfo(dtype).min
    z[0, 1] = float("nan")
    z[1, V - 1] = float("inf")
    z[2, V // 2] = float("nan")
    z[2, V // 2 + 1] = float("inf")
    z[3] = float("nan")
    z[4, 0] = float("nan")              # a row that does not count
    bad = np.arange(T) < 4
    tokens = np.full(T, 2, np.int32)
    tokens[4] = -1
    g, e = rng.normal(size=(2, T)).astype(np.float32)
    d_h = dev(e) if entropy else None
    heat = dev((0.5 + rng.random(T)).astype(np.float32))
    for dz in (lib().token_logprobs_backward(z, dev(tokens), dev(g), None, d_h),
               lib().token_logprobs_backward(z, dev(tokens), dev(0 * g), heat, dev(e)),
               lib().token_logprobs_backward(z, dev(tokens), dev(g), heat, d_h),
               lib().policy_loss_with_grad(z, dev(tokens), dev(g), dev(e),
                                           entropy=0.01 if entropy else None)[1]):
        dz = host(dz)
        assert np.isnan(dz[bad]).all()
        assert np.isfinite(dz[~bad]).all() and not dz[4].any()


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("t", [1e-45, 1e-42, 2e-39, 4e-39, 1e-38])
def test_log_probabilities_at_the_smallest_temperatures(T, V, t):
    """Where float32 holds the distance to the largest logit divided by the
    temperature, but not the temperature's inverse.  In the probabilities log2(e) /
    temperature counts as float32's largest number where it is beyond that."""
    note("smallest temperatures %d %d %g" % (T, V, t))
    t = float(np.float32(t))
    z = torch.zeros(T, V)
    z[:, 1:] = -1e30
    far = np.float32(t) * (10.0 ** np.linspace(5, 37, T))
    z[:, V // 2] = torch.from_numpy(-far.astype(np.float32))
    tokens = np.full(T, V // 2, np.int32)
    d = host(z[:, V // 2])
    u = d * min(np.log2(np.e) / t, float(np.finfo(np.float32).max))
    x = 2.0 ** u
    log_s = np.log1p(x)
    want, h = d / t - log_s, log_s - np.log(2) * u * x / (1 + x)
    # the exponent's product and the instruction are rounded; s = 1 + x to 2^-53, and
    # the logarithm's series leaves 1.2e-14
    err, log_err = U * (2 * np.abs(u) + 2) * x, 2.0 ** -53 + 1.2e-14
    for entropy in (False, True):
        got = lib().token_logprobs(dev(z.numpy()), dev(tokens), dev(np.full(T, t, np.float32)),
                                   entropy=entropy)
        lp = host(got[0] if entropy else got)
        assert np.all(np.abs(lp - want) <= err + log_err + U * np.abs(want))
        if entropy:
            assert np.all(np.abs(host(got[1]) - h) <= err * (1 + np.abs(u)) + log_err +
                          U * (4 * x + h))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("t,g", [(1e-42, 2.0), (1e-35, 65536.0), (1e-38, -1e3), (1e-30, 1e10),
                                 (1.0, 3e38), (1e-3, -3e36)])
def test_gradients_beyond_float32(T, V, dtype, t, g):
    """Where gradient / temperature is beyond float32, logits of probability 0 have
    gradient 0 all the same, and those that have a share of it are infinite."""
    note("gradients beyond float32 %d %d %s %g" % (T, V, dtype, t))
    rng = np.random.default_rng(V)
    t, g = float(np.float32(t)), float(np.float32(g))
    z = logits_of(rng, T, V, dtype)
    z[:, 4::5] = -float("inf")
    z[:, 3] = torch.finfo(dtype).min
    z[:, V // 2] = 1000.0               # a probability of 1
    z[3, 0] = 1000.0                    # two of 1/2
    tokens = np.full(T, V // 2, np.int32)
    tokens[1], tokens[2] = 1, 4         # of probability 0, masked
    p, one = np.zeros((2, T, V))
    p[:, V // 2] = 1.0
    p[3, [0, V // 2]] = 0.5
    one[np.arange(T), tokens] = 1.0
    want = (one - p) * (g / t)
    half = torch.finfo(dtype).eps / 2
    top = float(torch.finfo(dtype).max) * (1 + half)    # what is rounded to infinity
    for e in (None, 0.0, 1.0):
        d_h = None if e is None else dev(np.full(T, e, np.float32))
        got = host(lib().token_logprobs_backward(z, dev(tokens), dev(np.full(T, g, np.float32)),
                                                 dev(np.full(T, t, np.float32)), d_h))
        assert not np.isnan(got).any()
        rest = want == 0
        assert not got[rest].any()
        wild = np.abs(want) >= top
        assert np.array_equal(got[wild], np.copysign(np.inf, want[wild]))
        near = ~rest & ~wild
        # gradient, 1 / t, 1 / s and their products are rounded, in float32 or 64 bits
        err = (8 * 2.0 ** -24 + half) * np.abs(want[near])
        assert np.all(np.abs(got[near] - want[near]) <= err)


@pytest.mark.parametrize("q", [1e-6, 1e-5, 1e-4, 1e-3, 1e-2, 0.1, 0.3, 0.49, 0.51, 0.7, 1.0, 3.0])
@pytest.mark.parametrize("sign", [1, -1])
def test_divergence_from_a_near_reference(q, sign):
    """exp(q) - q - 1 of a small q is q^2 / 2, not what is left of q less q."""
    for V, dtype in ((4, torch.float32), (256, torch.float16), (65536, torch.bfloat16),
                     (131072, torch.float32)):
        note("divergence %g %d" % (sign * q, V))
        z = torch.zeros(1, V)
        ref = np.float32([-np.log(V) + sign * q])
        exact_q = float(ref[0]) + np.log(V)     # V is exact, and so is s
        x, want, n = exact_q, 0.0, 2
        term = x * x / 2
        while abs(term) > 1e-20 * want:         # for its tail to be of one size
            want += term
            n += 1
            term *= x / n
        one, zero = dev(np.ones(1, np.float32)), dev(np.zeros(1, np.float32))
        given = [dev(z.numpy(), dtype), dev(np.zeros(1, np.int32)), zero, zero, one, dev(ref)]
        for loss in (lib().policy_loss(*given, kl=1.0)[0],
                     lib().policy_loss_with_grad(*given, kl=1.0)[0]):
            # the logarithm is good to 1.2e-14, and the oracle's to 2^-52 log V; q is
            # rounded (2 U of q^2), beyond 1/2 the exponential less 1 and the
            # difference from q are (3 U of values up to 5 times the result, 8 at 3), below it 8
            # steps of a polynomial whose later ones count half and less
            err = (2 + 3 * 8) * U * want + (1.2e-14 + 2.0 ** -52 * np.log(V)) * abs(np.expm1(x))
            assert abs(float(loss) - want) <= err, (V, float(loss), want)
            assert float(loss) >= 0


# ------------------------------------------------------------------ temperatures

def representable(want, dtype):
    """Infinite where a type rounds a value to infinity."""
    info = torch.finfo(dtype)
    over = np.abs(want) >= float(info.max) * (1 + info.eps / 4)
    return np.where(over, np.copysign(np.inf, want), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(5, 7), (40, 257), (9, 2049), (3, 8191), (2, 50021), (300, 1000),
                                 (70, 5001), (97, 66001)])
@pytest.mark.parametrize("kl,entropy", [(0.0, None), (0.1, 0.05)])
def test_policy_with_temperatures(T, V, dtype, kl, entropy):
    """A temperature of each row's own, some that count as 1, in the call with the
    gradient and through autograd, with held ratios, divergence and entropies."""
    note("policy with temperatures %d %d %s %s" % (T, V, dtype, kl))
    rng = np.random.default_rng(T + 7 * V)
    z = logits_of(rng, T, V, dtype)
    heat = (0.4 + 1.3 * rng.random(T)).astype(np.float32)
    heat[::5] = rng.choice(np.float32([0, -2, np.nan, 1]), len(heat[::5]))
    tokens = tokens_of(rng, T, V, 0.1)
    lp = plain.rows(host(z), tokens, heat)[1]
    old, ref = (lp + 0.4 * rng.normal(size=(2, T))).astype(np.float32)
    adv, w = rng.normal(size=T).astype(np.float32), rng.random(T).astype(np.float32)
    w[rng.random(T) < 0.1] = 0.0
    up, bonus = 4.0, entropy or 0.0
    b = Bounds(host(z), tokens, heat, w)
    loss, lp, h, dz, g, e = plain.policy(host(z), tokens, old, adv, w, ref, heat, 0.2, 0.28, kl,
                                         bonus, up)
    err, dg = policy_bounds(b, old, adv, w, ref, kl, bonus, up)
    tol = b.grad(dtype, dz, g, e, dg)
    given = [dev(v) for v in (tokens, old, adv, w, ref, heat)]
    options = dict(clip=0.2, clip_high=0.28, kl=kl, entropy=entropy)
    both = lib().policy_loss_with_grad(z, *given, grad_loss=dev(np.float32([up])), **options)
    leaf = z.clone().requires_grad_()
    got = lib().policy_loss(leaf, *given, **options)
    got[0].backward(torch.tensor(up, device=z.device))
    within(host(both[1]), dz, tol, "gradient")
    within(host(leaf.grad), dz, tol, "gradient of autograd")
    for out in (both[:1] + both[2:], got, lib().policy_loss(z, *given, **options)):
        within(host(out[0]), loss, err + U * abs(loss), "loss")
        within(host(out[1]), lp, b.logprob, "logprobs")
        if entropy is not None:
            within(host(out[2]), h, b.entropy, "entropies")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(13, 333), (13, 9001), (13, 70001), (130, 66001)])
def test_gradients_at_any_temperature(T, V, dtype):
    """0, below and NaN as 1; very large and very small ones; infinity."""
    note("gradients at any temperature %d %d %s" % (T, V, dtype))
    rng = np.random.default_rng(V + 3)
    heat = np.resize(np.float32([0, -1, np.nan, 1e-3, 1e3, 1e30, np.inf, 1e-30, 1e-42, 3e38, 1e-38,
                                 -np.inf, 1]), T)
    z = logits_of(rng, T, V, dtype)
    z[:, 5] = -float("inf")
    z[:, 7] = 40.0                      # the largest of all rows, by more than any two are apart
    tokens = rng.integers(8, V, T).astype(np.int32)
    tokens[T // 2:] = 7
    g, e = rng.normal(size=(2, T)).astype(np.float32)
    b = Bounds(host(z), tokens, heat)
    lp, h = lib().token_logprobs(z, dev(tokens), dev(heat), entropy=True)
    within(host(lp), representable(b.lp, torch.float32), b.logprob, "logprobs")
    within(host(h), b.h, b.entropy, "entropies")
    for d_h in (None, e):
        want = plain.combine(b.counts, b.dlp, b.dh, g, d_h)
        got = host(lib().token_logprobs_backward(z, dev(tokens), dev(g), dev(heat), dev(d_h)))
        within(got, representable(want, dtype), b.grad(dtype, want, g, d_h), "gradient")
