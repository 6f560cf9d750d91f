"""Log probabilities of tokens, the policy loss and the preference loss on the
GPU against the plain 64-bit ones (bounds: loss_util.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gpu_util import device, note  # noqa: E402
from loss_util import TYPES, U, Bounds, dev, host, lib, logits_of, within  # noqa: E402
from oracle import losses as plain  # noqa: E402

pytestmark = pytest.mark.gpu

# one row to many, one token to a large vocabulary, odd sizes around every
# boundary of 8, 64, 256 elements, rows that split into slices and those that do not
SHAPES = [(1, 1), (3, 1), (5, 2), (4, 7), (3, 8), (2, 9), (7, 63), (5, 64), (3, 65), (33, 257),
          (1, 1000), (9, 2047), (2, 2049), (3, 4097), (2, 8191), (1, 32000), (2, 100003),
          (2100, 41), (2500, 130), (70, 5001),
          # around the sizes that a workgroup of 64, 128, 512 and 1024 threads holds
          (3, 1024), (2, 1025), (3, 2048), (2, 2049), (2, 4096), (3, 4097), (2, 8192), (2, 8193),
          (2, 16384), (2, 16385), (2, 32768), (2, 32769), (64, 40000), (70, 66000), (3, 65536),
          (2, 65537), (96, 70001), (2, 131072), (2, 131073), (1, 262144), (2, 300007)]


def tokens_of(rng, T, V, masked=0.2):
    """Some rows do not count; ids far outside the vocabulary among them."""
    a = rng.integers(0, V, T).astype(np.int32)
    out = rng.random(T) < masked
    a[out] = rng.choice([-1, V, V + 7, -2 ** 31, 2 ** 31 - 1], out.sum())
    return a


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", SHAPES)
def test_logprobs(T, V, dtype):
    note("logprobs %d %d %s" % (T, V, dtype))
    rng = np.random.default_rng(T * 1000 + V)
    heat = (0.3 + rng.random(T)).astype(np.float32) if V % 2 else None
    z = logits_of(rng, T, V, dtype)
    tokens = tokens_of(rng, T, V)
    b = Bounds(host(z), tokens, heat)
    got = lib().token_logprobs(z, dev(tokens), dev(heat))
    assert got.dtype == torch.float32 and got.shape == (T,)
    within(host(got), b.lp, b.logprob, "logprobs")
    lp, h = lib().token_logprobs(z, dev(tokens), dev(heat), entropy=True)
    within(host(lp), b.lp, b.logprob, "logprobs beside entropies")
    within(host(h), b.h, b.entropy, "entropies")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", SHAPES)
def test_logprobs_backward(T, V, dtype):
    note("logprobs backward %d %d %s" % (T, V, dtype))
    rng = np.random.default_rng(T * 1000 + V + 1)
    heat = (0.3 + rng.random(T)).astype(np.float32) if V % 2 == 0 else None
    z = logits_of(rng, T, V, dtype)
    tokens = tokens_of(rng, T, V)
    g, e = rng.normal(size=(2, T)).astype(np.float32)
    g[rng.random(T) < 0.1] = 0.0
    b = Bounds(host(z), tokens, heat)
    want = plain.combine(b.counts, b.dlp, b.dh, g, None)
    got = lib().token_logprobs_backward(z, dev(tokens), dev(g), dev(heat))
    assert got.dtype == dtype and got.is_contiguous()
    within(host(got), want, b.grad(dtype, want, g), "gradient")
    want = plain.combine(b.counts, b.dlp, b.dh, g, e)
    got = lib().token_logprobs_backward(z, dev(tokens), dev(g), dev(heat), dev(e))
    within(host(got), want, b.grad(dtype, want, g, e), "gradient with entropies")


def policy_inputs(rng, T, V, dtype, masked=0.2):
    z = logits_of(rng, T, V, dtype)
    tokens = tokens_of(rng, T, V, masked / 2)
    weights = rng.random(T).astype(np.float32)
    weights[rng.random(T) < masked / 2] = 0.0
    lp = plain.rows(host(z), tokens)[1]
    old = (lp + 0.4 * rng.normal(size=T)).astype(np.float32)
    ref = (lp + 0.4 * rng.normal(size=T)).astype(np.float32)
    adv = rng.normal(size=T).astype(np.float32)
    adv[rng.random(T) < 0.1] = 0.0
    return z, tokens, old, adv, weights, ref


def policy_bounds(b, old, adv, w, ref, kl, entropy, up=1.0):
    """(loss, gradient in the log probability) may be off by this: the ratio by
    the log probability's error and 4 U (its difference, exp), the divergence by
    expm1's slope times that error; products 3 U."""
    w = np.where(b.counts, w, 0.0)
    with np.errstate(over="ignore"):
        size = np.exp(b.lp - old) * np.abs(adv)
        q = np.exp(ref - b.lp) if kl else np.zeros_like(b.lp)
    err = b.logprob
    dg = np.abs(w * up) * (size * (err + 7 * U) + kl * (q * err + 4 * U * (q + 1)))
    loss = np.abs(w) * (size * (err + 7 * U) + kl * (np.abs(q - 1) * err + 5 * U * (q + 1)) +
                        abs(entropy) * (b.entropy + 3 * U * b.h))
    return loss.sum(), dg


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(1, 1), (5, 7), (3, 64), (40, 257), (9, 2049), (3, 8191),
                                 (2, 50021), (2200, 33), (300, 1000), (70, 5001)])
@pytest.mark.parametrize("kl,entropy", [(0.0, None), (0.1, None), (0.1, 0.05)])
def test_policy(T, V, dtype, kl, entropy):
    note("policy %d %d %s %s %s" % (T, V, dtype, kl, entropy))
    rng = np.random.default_rng(T + V)
    z, tokens, old, adv, w, ref = policy_inputs(rng, T, V, dtype)
    up = 4.0
    b = Bounds(host(z), tokens, None, w)
    bonus = entropy or 0.0
    loss, lp, h, dz, g, e = plain.policy(host(z), tokens, old, adv, w, ref, None, 0.2, 0.28, kl,
                                         bonus, up)
    err, dg = policy_bounds(b, old, adv, w, ref, kl, bonus, up)
    given = [dev(v) for v in (tokens, old, adv, w, ref)]
    options = dict(clip=0.2, clip_high=0.28, kl=kl, entropy=entropy)
    got = lib().policy_loss(z, *given, **options)
    assert len(got) == (2 if entropy is None else 3) and got[0].shape == ()
    within(host(got[0]), loss, err + U * abs(loss), "loss")
    within(host(got[1]), lp, b.logprob, "logprobs")
    if entropy is not None:
        within(host(got[2]), h, b.entropy, "entropies")
    both = lib().policy_loss_with_grad(z, *given, grad_loss=dev(np.float32([up])), **options)
    within(host(both[0]), loss, err + U * abs(loss), "loss beside the gradient")
    within(host(both[2]), lp, b.logprob, "logprobs beside the gradient")
    if entropy is not None:
        within(host(both[3]), h, b.entropy, "entropies beside the gradient")
    within(host(both[1]), dz, b.grad(dtype, dz, g, e, dg), "gradient")
    # through autograd
    leaf = z.clone().requires_grad_()
    loss2 = lib().policy_loss(leaf, *given, **options)[0]
    loss2.backward(torch.tensor(up, device=device()))
    within(host(loss2), loss, err + U * abs(loss), "loss with a graph")
    within(host(leaf.grad), dz, b.grad(dtype, dz, g, e, dg), "gradient of autograd")


def test_policy_defaults():
    """Without weights a row weighs 1 / rows; without kl the reference is not read."""
    rng = np.random.default_rng(5)
    z, tokens, old, adv, _, ref = policy_inputs(rng, 37, 501, torch.float32)
    loss, lp, _, dz, g, _ = plain.policy(host(z), tokens, old, adv)
    b = Bounds(host(z), tokens)
    err, dg = policy_bounds(b, old, adv, np.full(37, 1 / 37), ref, 0.0, 0.0)
    got = lib().policy_loss_with_grad(z, dev(tokens), dev(old), dev(adv),
                                      ref_logprobs=dev(ref * np.float32(np.nan)))
    within(host(got[0]), loss, err + 2 * U * abs(loss), "loss")
    within(host(got[1]), dz, b.grad(torch.float32, dz, g, None, dg + U * np.abs(g)), "gradient")


def preference_bounds(b, at, sums, margins, w, beta, kind, average, up, known=False):
    """(loss, logprobs, margins, gradient in the log probabilities): a sum is off
    by those of its rows, the margin by beta times both of its sums'."""
    P = len(margins)
    size = [max(1, b.counts[at[q]:at[q + 1]].sum()) if average else 1 for q in range(2 * P)]
    err = np.array([b.logprob[at[q]:at[q + 1]].sum() / size[q] for q in range(2 * P)])
    dh = beta * (err[:P] + err[P:]) + U * np.abs(margins)
    with np.errstate(invalid="ignore"):
        curve = {"sigmoid": 0.25, "hinge": 0.0, "squared": 2 / beta ** 2}[kind]
        slope = {"sigmoid": np.ones(P), "hinge": np.ones(P),
                 "squared": 2 * np.abs(margins - 0.5) / beta ** 2}[kind]
    loss = (np.abs(w) * (slope * dh + curve * dh ** 2)).sum()
    dg = np.zeros(len(b.lp))
    for i in range(P):
        for q in (i, P + i):
            dg[at[q]:at[q + 1]] = up * beta / size[q] * abs(w[i]) * (curve * dh[i] +
                                                                     2 * U * slope[i])
    return loss, err + U * np.abs(sums), dh, dg


def sequences(rng, T, pairs):
    """Ragged sequences, an empty one among them, rows before and behind them."""
    cut = np.sort(rng.integers(T // 8, T + 1 - T // 8, 2 * pairs + 1))
    if pairs > 1:
        cut[2] = cut[1]
    return cut.astype(np.int64)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V,P", [(2, 5, 1), (16, 33, 2), (40, 1000, 3), (6, 40001, 1),
                                   (2300, 70, 5), (200, 257, 40)])
@pytest.mark.parametrize("kind,average", [("sigmoid", False), ("sigmoid", True),
                                          ("hinge", False), ("squared", True)])
def test_preference(T, V, P, dtype, kind, average):
    note("preference %d %d %d %s %s %s" % (T, V, P, dtype, kind, average))
    rng = np.random.default_rng(T + V + P)
    z = logits_of(rng, T, V, dtype)
    tokens = tokens_of(rng, T, V)
    at = sequences(rng, T, P)
    beta, up, smoothing = 0.25, 8.0, 0.1 if kind == "sigmoid" else 0.0
    b = Bounds(host(z), tokens)
    sums = plain.preference(host(z), tokens, at, average=average)[1]
    ref = (sums + 2 * rng.normal(size=2 * P)).astype(np.float32)
    w = rng.random(P).astype(np.float32)
    if P > 2:
        w[1] = 0.0
    loss, sums, margins, dz, g = plain.preference(host(z), tokens, at, ref, w, beta, kind,
                                                  smoothing, 0.125, average, up)
    err, dsum, dh, dg = preference_bounds(b, at, sums, margins, w, beta, kind, average, up)
    options = dict(beta=beta, kind=kind, smoothing=smoothing, margin=0.125, average=average)
    given = [dev(v) for v in (tokens, at, ref, w)]
    for got in (lib().preference_loss(z, *given, **options),
                lib().preference_loss_with_grad(z, *given, grad_loss=dev(np.float32([up])),
                                                **options)):
        within(host(got[0]), loss, err + 4 * U * abs(loss), "loss")
        within(host(got[-2]), sums, dsum, "logprobs")
        within(host(got[-1]), margins, dh, "margins")
    within(host(got[1]), dz, b.grad(dtype, dz, g, None, dg), "gradient")
    leaf = z.clone().requires_grad_()
    lib().preference_loss(leaf, *given, **options)[0].backward(torch.tensor(up, device=device()))
    within(host(leaf.grad), dz, b.grad(dtype, dz, g, None, dg), "gradient of autograd")


# --------------------------------------------------- layouts and odd values

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,stride,shift", [(1000, 1000, 1), (1000, 1003, 0), (1001, 1001, 3),
                                            (5003, 6000, 5), (40007, 40009, 1)])
def test_strides_and_alignment(V, stride, shift, dtype):
    """Rows at any element's address; what lies between them (NaN) and in the
    output's gaps is neither read nor written."""
    note("strides %d %d %d %s" % (V, stride, shift, dtype))
    rng = np.random.default_rng(V + stride)
    T = 5
    z = logits_of(rng, T, V, dtype, stride=stride, shift=shift)
    tokens = np.array([0, V - 1, V // 2, -1, 7], np.int32)
    g, e = rng.normal(size=(2, T)).astype(np.float32)
    b = Bounds(host(z), tokens)
    lp, h = lib().token_logprobs(z, dev(tokens), entropy=True)
    within(host(lp), b.lp, b.logprob, "logprobs")
    within(host(h), b.h, b.entropy, "entropies")
    want = plain.combine(b.counts, b.dlp, b.dh, g, e)
    space = torch.full((T, stride + 5), 7.0, dtype=dtype, device=device())
    out = space[:, 2:2 + V]
    got = lib().token_logprobs_backward(z, dev(tokens), dev(g), None, dev(e), out=out)
    assert got is out
    within(host(out), want, b.grad(dtype, want, g, e), "gradient")
    assert bool((space[:, :2] == 7).all()) and bool((space[:, 2 + V:] == 7).all())
    # in place of the logits
    got = lib().token_logprobs_backward(z, dev(tokens), dev(g), None, dev(e), out=z)
    assert torch.equal(z, out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [9, 700, 9001, 70001])
def test_masks_and_lowest_values(V, dtype):
    """Rows masked by -infinity or by the type's lowest value: all of them, all
    but one, the token itself; and the largest values of the type."""
    note("masks %d %s" % (V, dtype))
    rng = np.random.default_rng(V)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    z = logits_of(rng, 11, V, dtype)
    z[0] = -float("inf")
    z[1] = low
    z[2] = -float("inf")
    z[2, V // 2] = 3.0
    z[3] = low
    z[3, V // 2] = 1.0
    z[4, 1::2] = -float("inf")
    z[5, 1::2] = low
    z[6] = high
    z[7, 0] = high
    z[8] = low
    z[8, V // 2] = high
    z[9, V // 2] = -float("inf")      # the token
    z[10] = 0.0
    tokens = np.full(11, V // 2, np.int32)
    tokens[[4, 5]] = 2 * (V // 4)
    heat = np.ones(11, np.float32)
    g, e = rng.normal(size=(2, 11)).astype(np.float32)
    b = Bounds(host(z), tokens, heat)
    for t in (None, dev(heat)):
        lp, h = lib().token_logprobs(z, dev(tokens), t, entropy=True)
        within(host(lp), b.lp, b.logprob, "logprobs")
        within(host(h), b.h, b.entropy, "entropies")
        for d_h in (None, e):
            want = plain.combine(b.counts, b.dlp, b.dh, g, d_h)
            got = lib().token_logprobs_backward(z, dev(tokens), dev(g), t, dev(d_h))
            within(host(got), want, b.grad(dtype, want, g, d_h), "gradient")
    assert np.isneginf(host(lp)[0]) and np.isneginf(host(lp)[9])
    assert not host(got)[0].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [9, 9001, 70001])
def test_nan_and_infinity(V, dtype):
    """NaN or +infinity in a row that counts shows; in rows that do not count, in
    rows of weight 0 and without an upstream gradient it does not."""
    note("nan %d %s" % (V, dtype))
    rng = np.random.default_rng(V + 1)
    z = logits_of(rng, 7, V, dtype)
    z[0, V - 1] = float("nan")
    z[1, 3] = float("inf")
    z[2] = float("nan")
    z[3] = float("nan")
    z[4] = float("inf")
    z[5, 2] = float("nan")
    tokens = np.array([1, 1, 1, -1, V, 1, 1], np.int32)
    bad = np.array([True, True, True, False, False, True, False])
    lp, h = lib().token_logprobs(z, dev(tokens), entropy=True)
    assert np.array_equal(np.isnan(host(lp)), bad) and np.array_equal(np.isnan(host(h)), bad)
    g = np.ones(7, np.float32)
    g[5] = 0.0
    dz = host(lib().token_logprobs_backward(z, dev(tokens), dev(g)))
    assert np.isnan(dz[:3]).all() and not dz[3:6].any() and np.isfinite(dz[6]).all()
    w = np.array([0, 0, 0, 1, 1, 0, 1], np.float32)
    zero = np.zeros(7, np.float32)
    loss, dz, lp = lib().policy_loss_with_grad(z, dev(tokens), dev(zero), dev(zero + 1), dev(w))
    assert np.isfinite(host(loss)) and not host(dz)[:6].any() and np.isfinite(host(dz)).all()
    assert not host(lp)[:6].any()
    # a row of weight NaN counts
    w[0] = np.nan
    loss, dz, lp = lib().policy_loss_with_grad(z, dev(tokens), dev(zero), dev(zero + 1), dev(w))
    assert np.isnan(host(loss)) and np.isnan(host(dz)[0]).all()


def test_temperatures():
    """0, below and NaN as 1; very large and very small ones; infinity."""
    note("temperatures")
    rng = np.random.default_rng(7)
    heat = np.array([0, -1, np.nan, 1e-3, 1e3, 1e30, np.inf, 1e-30, 1e-42, 3e38], np.float32)
    T, V = len(heat), 333
    for dtype in TYPES:
        z = logits_of(rng, T, V, dtype)
        z[:, 5] = -float("inf")
        tokens = rng.integers(6, V, T).astype(np.int32)
        tokens[8] = int(z[8].argmax())
        b = Bounds(host(z), tokens, heat)
        lp, h = lib().token_logprobs(z, dev(tokens), dev(heat), entropy=True)
        # at 1e-42 an inverse that float32 holds stands for it: the row's
        # largest logit has probability 1 either way (equal ones share it)
        within(host(lp), b.lp, b.logprob, "logprobs")
        usual = np.arange(T) != 7
        within(host(h)[usual], b.h[usual], b.entropy[usual], "entropies")


def test_ratios_out_of_range():
    """An advantage of 0 has no term, whatever the ratio; a ratio beyond
    float32 is held for a positive advantage and infinite for a negative one."""
    z = torch.zeros(5, 4, device=device())
    tokens = dev(np.zeros(5, np.int32))
    old = dev(np.float32([-np.inf, -200, -200, 200, -np.inf]))
    adv = dev(np.float32([0, 1, -1, 1, np.nan]))
    loss, dz, lp = lib().policy_loss_with_grad(z[:2], tokens[:2], old[:2], adv[:2])
    assert float(loss) == pytest.approx(-0.6) and not host(dz).any()
    loss, dz, lp = lib().policy_loss_with_grad(z[2:3], tokens[2:3], old[2:3], adv[2:3])
    assert np.isposinf(host(loss))
    loss, dz, lp = lib().policy_loss_with_grad(z[3:4], tokens[3:4], old[3:4], adv[3:4])
    assert float(loss) == 0 and not host(dz).any()
    loss, dz, lp = lib().policy_loss_with_grad(z[4:], tokens[4:], old[4:], adv[4:])
    assert np.isnan(host(loss)) and np.isnan(host(dz)).all()


def test_offsets_out_of_order():
    """Offsets outside the rows or decreasing: the largest so far, within them."""
    rng = np.random.default_rng(8)
    z = logits_of(rng, 12, 50, torch.float32)
    tokens = rng.integers(0, 50, 12).astype(np.int32)
    for at in ([-5, 3, 2, 99, 4], [13, 14, 15, 16, 17], [0, 0, 0, 0, 0], [2, 2, 12, 12, 12],
               [2 ** 40, 0, 1, 2, 3], [-2 ** 62, 4, 2 ** 62, 5, 6]):
        at = np.array(at, np.int64)
        loss, sums, margins, dz, g = plain.preference(host(z), tokens, at)
        b = Bounds(host(z), tokens)
        got = lib().preference_loss_with_grad(z, dev(tokens), dev(at))
        err, dsum, dh, dg = preference_bounds(b, plain.starts(at, 12), sums, margins,
                                              np.full(2, 0.5), 0.1, "sigmoid", False, 1.0)
        within(host(got[0]), loss, err + 4 * U * abs(loss), "loss")
        within(host(got[1]), dz, b.grad(torch.float32, dz, g, None, dg), "gradient")
        within(host(got[2]), sums, dsum, "logprobs")


def test_pairs_of_infinite_log_probability():
    """A preferred answer of probability 0 has an infinite loss, the other one of
    a pair none."""
    z = torch.zeros(4, 3, device=device())
    z[0, 1] = -float("inf")
    tokens = dev(np.ones(4, np.int32))
    at = dev(np.array([0, 2, 4]))
    loss, dz, lp, h = lib().preference_loss_with_grad(z, tokens, at)
    assert np.isposinf(host(loss)) and np.isneginf(host(h)).all() and np.isfinite(host(dz)).all()
    at = dev(np.array([0, 0, 2]))
    loss, dz, lp, h = lib().preference_loss_with_grad(z, tokens, at, kind="hinge")
    assert float(loss) == 0 and np.isposinf(host(h)).all() and not host(dz).any()
    # a pair that has no weight
    loss, dz, lp, h = lib().preference_loss_with_grad(z, tokens, dev(np.array([0, 2, 4])),
                                                      weights=dev(np.float32([0])))
    assert float(loss) == 0 and not host(dz).any()


def test_empty():
    z = torch.zeros(0, 9, device=device())
    none = torch.zeros(0, device=device())
    ids = torch.zeros(0, dtype=torch.int32, device=device())
    assert lib().token_logprobs(z, ids).shape == (0,)
    assert lib().token_logprobs_backward(z, ids, none).shape == (0, 9)
    loss, dz, lp = lib().policy_loss_with_grad(z, ids, none, none)
    assert float(loss) == 0 and dz.shape == (0, 9)
    at = torch.zeros(5, dtype=torch.int64, device=device())
    loss, dz, lp, h = lib().preference_loss_with_grad(z, ids, at)
    assert float(loss) == pytest.approx(np.log(2)) and lp.tolist() == [0] * 4
    loss, dz, counts = lib().balance_loss_with_grad(z, torch.zeros(0, 2, dtype=torch.int32,
                                                                   device=device()))
    assert float(loss) == 0 and counts.tolist() == [0] * 9


def test_rows_past_two_gigaelements():
    """Rows whose elements start beyond 2^31 of the first."""
    note("far rows")
    V, stride = 5000, 5000 + (1 << 30)
    space = torch.zeros(3 * stride, dtype=torch.float16, device=device())
    z = space.view(3, stride)[:, :V]
    rng = np.random.default_rng(9)
    z.copy_(dev(rng.normal(size=(3, V)).astype(np.float32)))
    tokens = np.array([5, 4999, 17], np.int32)
    b = Bounds(host(z), tokens)
    within(host(lib().token_logprobs(z, dev(tokens))), b.lp, b.logprob, "logprobs")
    g = np.float32([1, -2, 3])
    want = plain.combine(b.counts, b.dlp, b.dh, g, None)
    got = lib().token_logprobs_backward(z, dev(tokens), dev(g), out=z)
    within(host(got), want, b.grad(torch.float16, want, g), "gradient")
