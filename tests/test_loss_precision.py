"""The bounds of loss_precision.py on the CPU: a model of the kernels' arithmetic
is within them; one with float32 sums, or without the scale's second term, is not."""
import numpy as np
import pytest
import torch

import loss_precision as lp


def model(z, tokens, t, second=True, sums=np.float64, threads=256, group=8):
    """Log probabilities by float32 differences, products and exponentials.  sums:
    the type in which a thread adds its own, `group` at a time by halves."""
    z = z.float().numpy()
    top = z[np.arange(len(z)), tokens.numpy()][:, None]
    k = np.log2(np.e) / float(t)
    hi = np.float32(k)
    if float(hi) > k:
        hi = np.nextafter(hi, np.float32(0))
    low = np.float32(k - float(hi)) if second else np.float32(0)
    d = z - top
    # (the product and the sum are exact in binary64, then rounded once)
    u = (d.astype(np.float64) * float(hi) + d.astype(np.float64) * float(low)).astype(np.float32)
    x = np.exp2(u.astype(np.float64)).astype(np.float32)
    pad = -len(x[0]) % (threads * group)
    x = np.pad(x, ((0, 0), (0, pad))).reshape(len(x), -1, threads, group)
    if sums is np.float32:
        while x.shape[3] > 1:
            x = x[..., :x.shape[3] // 2] + x[..., x.shape[3] // 2:]
    total = np.zeros((len(x), threads), sums)
    for i in range(x.shape[1]):
        for j in range(x.shape[3]):
            total = total + x[:, i, :, j].astype(sums)
    while total.shape[1] > 1:
        total = total[:, :total.shape[1] // 2] + total[:, total.shape[1] // 2:]
    return (-np.log(total[:, 0].astype(np.float64))).astype(np.float32)


def errors(got, b):
    return np.abs(got - b.logprob)


@pytest.mark.parametrize("V,away", [(8000, 7.0), (32000, 5.0), (32000, 7.0), (131072, 7.0)])
def test_float32_sums_are_not_within(V, away):
    g = torch.Generator()
    g.manual_seed(V)
    z, tokens = lp.standing_out(g, 12, V, torch.float32, away)
    b = lp.Rest(z, tokens)
    bound = b.of_logprob(b.of_rest())
    assert np.all(errors(model(z, tokens, 1.0), b) <= bound)
    assert np.any(errors(model(z, tokens, 1.0, sums=np.float32), b) > bound)


@pytest.mark.parametrize("V", [500, 8000, 32000])
def test_a_scale_without_its_second_term_is_not_within(V):
    g = torch.Generator()
    g.manual_seed(V)
    z, tokens = lp.standing_out(g, 12, V, torch.float32, 7.0)
    t = lp.awkward_temperature()
    z *= float(t)
    b = lp.Rest(z, tokens, float(t))
    bound = b.of_logprob(b.of_one_sign(2))
    assert np.all(errors(model(z, tokens, t), b) <= bound)
    assert np.all(errors(model(z, tokens, t, second=False), b) > bound)


def test_the_rest_by_hand():
    z = torch.tensor([[0.0, -1.0, -2.0]])
    b = lp.Rest(z, torch.tensor([0], dtype=torch.int32), 2.0)
    rest = np.exp(-0.5) + np.exp(-1.0)
    assert np.allclose(b.rest, rest) and np.allclose(b.logprob, -np.log(1 + rest))
    assert np.allclose(b.gradient, (1 - 1 / (1 + rest)) / 2)
    assert np.allclose(b.far, 0.5 * np.exp(-0.5) + np.exp(-1.0))
