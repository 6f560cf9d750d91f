"""Results near 0: log probabilities and gradients of tokens that stand out, in
every way of launching, against 64 bits (bounds: loss_precision.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gpu_util import device, note  # noqa: E402
from loss_precision import LOG, U, Rest, awkward_temperature, standing_out  # noqa: E402
from loss_util import SMALL, TYPES, host, lib  # noqa: E402

pytestmark = pytest.mark.gpu


def rows(T, V, dtype, away, spread=1.0):
    g = torch.Generator(device=device())
    g.manual_seed(T + V)
    return standing_out(g, T, V, dtype, away, spread)


# rows in workgroups of 64, 128, 512 and 1024 threads; shared by slices; results of
# long rows in one workgroup's turns; gradients of rows that it holds and of longer ones
SHAPES = [(40, 500), (40, 3000), (20, 8000), (20, 32000), (70, 40001), (6, 131072), (100, 131072),
          (520, 131072)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("away", [4.0, 7.0, 10.0])
def test_tokens_that_stand_out(T, V, dtype, away):
    note("standing out %d %d %s %g" % (T, V, dtype, away))
    z, tokens = rows(T, V, dtype, away)
    b = Rest(z, tokens)
    of_rest = b.of_rest()
    bound = b.of_logprob(of_rest)
    old = torch.full((T,), -0.001, device=device())
    up = torch.full((T,), 1024.0, device=device())
    at = torch.arange(T, device=device()), tokens.long()
    results = [lib().token_logprobs(z, tokens), lib().token_logprobs(z, tokens, entropy=True)[0],
               lib().policy_loss_with_grad(z, tokens, old, up)[2],
               lib().policy_loss_with_grad(z, tokens, old, up, entropy=0.01)[2]]
    for got in results:
        assert np.all(np.abs(host(got) - b.logprob) <= bound)
    # its gradient: 1 - 1 / s in binary64, by the scale's first term alone with
    # entropies (2^-26 of x there); products and the conversion are rounded
    half = torch.finfo(dtype).eps / 2
    zero = torch.zeros(T, device=device())
    for entropies, more in ((None, 0.0), (zero, U * b.far)):
        got = host(lib().token_logprobs_backward(z, tokens, up, None, entropies)[at])
        want = 1024.0 * b.gradient
        err = 1024.0 * ((of_rest + more) / (1 + b.rest) + LOG) + (half + 4 * U) * want
        assert np.all(np.abs(got - want) <= err * (1 + half) + SMALL[dtype])


# (chunks of a row that a thread takes one after another)
@pytest.mark.parametrize("T,V,chunks", [(40, 500, 1), (20, 8000, 2), (64, 32000, 2),
                                        (6, 131072, 1), (100, 131072, 8)])
@pytest.mark.parametrize("entropy", [False, True])
def test_errors_do_not_add_up(T, V, chunks, entropy):
    """At a temperature whose scale float32 rounds by nearly an ulp, errors over a
    row's exponentials stay those of the instruction."""
    note("one sign %d %d" % (T, V))
    t = awkward_temperature()
    z, tokens = rows(T, V, torch.float32, 7.0)
    z *= float(t)
    b = Rest(z, tokens, float(t))
    heat = torch.full((T,), float(t), device=device())
    bound = b.of_logprob(b.of_one_sign(chunks))
    old = torch.full((T,), -0.001, device=device())
    got = (lib().token_logprobs(z, tokens, heat, entropy=True)[0] if entropy else
           lib().token_logprobs(z, tokens, heat))
    if chunks < 8:      # (those of (100, 131072) are made by more than eight)
        assert np.all(np.abs(host(got) - b.logprob) <= bound)
    got = lib().policy_loss_with_grad(z, tokens, old, old, temperature=heat,
                                      entropy=0.01 if entropy else None)[2]
    assert np.all(np.abs(host(got) - b.logprob) <= bound)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(4000, 500), (3000, 2000), (2000, 8000), (600, 32000)])
def test_sums_over_many_rows(T, V, dtype):
    """Of two sequences, each off by what its rows are off by in one direction."""
    note("sums of rows %d %d %s" % (T, V, dtype))
    z, tokens = rows(T, V, dtype, 5.0)
    b = Rest(z, tokens)
    cut = [0, T // 3, T]
    offsets = torch.tensor(cut, device=device())
    got = lib().preference_loss(z, tokens, offsets)[1]
    for q in range(2):
        mine = slice(cut[q], cut[q + 1])
        # at most four chunks; a type's equal logits round alike: their roundings
        # count as of one sign here
        err = (U * (2 * b.far + 2 * (4 + 3) * b.rest) + LOG)[mine].sum()
        want = b.logprob[mine].sum()
        assert abs(float(got[q]) - want) <= err + U * abs(want)
