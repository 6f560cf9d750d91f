"""Log probabilities of tokens that stand out, and how near their results have to
be: where a row's largest logit is the token's, s = 1 + rest with the rest of the
exponentials, log p = -log(1 + rest) and its gradient g / t * rest / (1 + rest).

With U = 2^-24 and x = (m - z) / t, an exponential of the rest is off by

* its difference and its product with log2(e) / t, each rounded once: 2 U x of its
  value.  The scale's own error is 2^-48, as it is a sum of two (or the sum is
  corrected for the second), and does not count;
* the instruction, good to an ulp: 2 U;
* each time that what it was added to is brought to another largest logit, the
  same for that factor: the distances add up to x, so 2 U more for each of K times.
  Within a thread the chunks of its row come one after another, C of them, then
  waves, workgroup and slices join: K = C + 2.

That is (2 x + 2 (1 + K)) U.  The largest one is 1 exactly, and sums are in
binary64: 2^-53 and the logarithm's 1.2e-14 are all that they add.  The roundings
of differences and products go either way, so that over a row's many exponentials
only the instruction's 2 (1 + K) U may be of one sign, and the others add up like
independent ones: sqrt(2 / 3) U x each.
"""
import numpy as np
import torch

U = 2.0 ** -24
CHUNKS = 16     # of a row by one thread, at most, in what is tested here
LOG = 2.0 ** -53 + 1.2e-14


def standing_out(generator, T, V, dtype, away, spread=1.0):
    """Logits whose token has exp(-away) of its weight beside it, and the tokens."""
    device = generator.device
    z = torch.randn(T, V, generator=generator, device=device) * spread
    tokens = (torch.rand(T, generator=generator, device=device) * V).long().clamp_(max=V - 1)
    z.scatter_(1, tokens[:, None], float("-inf"))
    level = torch.logsumexp(z.double(), dim=1) + away
    z.scatter_(1, tokens[:, None], level.float()[:, None])
    return z.to(dtype), tokens.to(torch.int32)


class Rest:
    """What log probabilities of such rows are, in 64 bits, and their bounds."""

    def __init__(self, z, tokens, t=1.0):
        at = tokens.long()[:, None]
        x = (z.double().gather(1, at) - z.double()) / t
        assert bool((x >= 0).all())
        e = torch.exp(-x).scatter_(1, at, 0.0)
        cpu = lambda v: v.cpu().numpy()  # noqa: E731
        self.rest, self.far = cpu(e.sum(1)), cpu((e * x).sum(1))
        self.noise = U * np.sqrt(2.0 / 3.0) * cpu(((e * x) ** 2).sum(1).sqrt())
        self.logprob = -np.log1p(self.rest)
        self.gradient = self.rest / (1.0 + self.rest) / t

    def of_rest(self, chunks=CHUNKS):
        """Of the rest, at most."""
        return U * (2 * self.far + 2 * (chunks + 3) * self.rest)

    def of_one_sign(self, chunks):
        """Of the rest, as far as roundings do not cancel, and six deviations of
        those that do."""
        return U * 2 * (chunks + 3) * self.rest + 6 * self.noise

    def of_logprob(self, rest):
        return rest / (1 + self.rest) + U * np.abs(self.logprob) + LOG


def awkward_temperature():
    """A temperature whose scale log2(e) / t lies just below a float32: the float
    below it alone is off by nearly 2^-23 of it."""
    t = np.float32(1.4426) + np.arange(400, dtype=np.float32) * np.float32(2.0 ** -23)
    k = np.log2(np.e) / t.astype(np.float64)
    t, k = t[(k > 1.0) & (k < 1.001)], k[(k > 1.0) & (k < 1.001)]
    hi = np.floor(k * 2.0 ** 23) / 2.0 ** 23
    return t[np.argmax((k - hi) / k)]
