"""The plain 64-bit losses against small hand-made cases and central
differences (CPU)."""
import numpy as np
import pytest

from oracle import losses as plain


def differences(f, z, step=1e-6):
    out = np.zeros_like(z)
    for at in np.ndindex(*z.shape):
        up, down = z.copy(), z.copy()
        up[at] += step
        down[at] -= step
        out[at] = (f(up) - f(down)) / (2 * step)
    return out


def close(got, want, tol=2e-8):
    """Differences of step 1e-6 in 64 bits: 1e-16 / 1e-6 of rounding and 1e-12
    times a third derivative of cancellation, with values of a few units."""
    assert np.abs(got - want).max() <= tol * max(1.0, np.abs(want).max())


def test_log_softmax_by_hand():
    y = plain.log_softmax([0.0, np.log(3.0), -np.inf])
    assert np.allclose(y[:2], np.log([0.25, 0.75])) and y[2] == -np.inf
    assert np.allclose(plain.log_softmax([0.0, 2.0], 2.0),
                       [-np.log(1 + np.e), 1 - np.log(1 + np.e)])
    assert np.isneginf(plain.log_softmax([-np.inf, -np.inf])).all()
    assert np.isnan(plain.log_softmax([1.0, np.nan])).all()
    assert np.allclose(plain.log_softmax([1.0, 5.0, -np.inf], np.inf)[:2], -np.log(2))


def test_rows_that_do_not_count():
    z = np.zeros((4, 3))
    counts, lp, h, dlp, dh = plain.rows(z, [0, -1, 3, 2], weights=[1, 1, 1, 0])
    assert counts.tolist() == [True, False, False, False]
    assert lp[0] == pytest.approx(-np.log(3)) and h[0] == pytest.approx(np.log(3))
    assert not lp[1:].any() and not h[1:].any() and not dlp[1:].any() and not dh[1:].any()


@pytest.mark.parametrize("temperature", [None, np.array([0.5, 1.7, 0.0])])
def test_gradients_of_rows(temperature):
    rng = np.random.default_rng(0)
    z = rng.normal(size=(3, 7))
    tokens = [2, -1, 6]
    g, e = rng.normal(size=3), rng.normal(size=3)

    def f(z):
        _, lp, h, _, _ = plain.rows(z, tokens, temperature)
        return (g * lp + e * h).sum()

    counts, _, _, dlp, dh = plain.rows(z, tokens, temperature)
    close(differences(f, z), plain.combine(counts, dlp, dh, g, e))


def test_policy_gradient():
    rng = np.random.default_rng(1)
    T, V = 24, 5
    z = rng.normal(size=(T, V))
    tokens = rng.integers(-1, V, T)
    lp = plain.rows(z, tokens)[1]
    old, ref = lp + 0.5 * rng.normal(size=T), lp + 0.5 * rng.normal(size=T)
    adv, w = rng.normal(size=T), np.where(rng.random(T) < 0.2, 0.0, rng.random(T))

    def f(z):
        return plain.policy(z, tokens, old, adv, w, ref, None, 0.2, 0.3, 0.1, 0.05)[0]

    got = plain.policy(z, tokens, old, adv, w, ref, None, 0.2, 0.3, 0.1, 0.05, up=2.0)
    close(2.0 * differences(f, z), got[3])
    # some ratios are held, on both sides
    assert (got[4] == 0).any() and (got[4] != 0).any()


def test_policy_by_hand():
    # two tokens of probability 1/2; ratios 2 and 1/2
    z = np.zeros((4, 2))
    old = np.log([0.25, 0.25, 1.0, 1.0])
    loss, lp, h, dz, g, e = plain.policy(z, [0, 0, 0, 0], old, [1.0, -1.0, 1.0, -1.0],
                                         weights=np.ones(4), clip=0.2)
    # held at 1.2; free -2; free 1/2; held at -0.8
    assert loss == pytest.approx(-1.2 + 2.0 - 0.5 + 0.8)
    assert np.allclose(g, [0.0, 2.0, -0.5, 0.0])


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
@pytest.mark.parametrize("average", [False, True])
def test_preference_gradient(kind, average):
    rng = np.random.default_rng(2)
    T, V = 20, 4
    z = rng.normal(size=(T, V))
    tokens = rng.integers(-1, V, T)
    offsets = [1, 5, 5, 9, 14, 16, 19]
    ref, w = rng.normal(size=6), np.array([1.0, 0.0, 0.5])
    args = (tokens, offsets, ref, w, 0.4, kind, 0.1 if kind == "sigmoid" else 0.0, 0.2, average)
    got = plain.preference(z, *args)
    close(differences(lambda z: plain.preference(z, *args)[0], z), got[3])
    assert not got[3][0].any() and not got[3][19].any()


def test_offsets_that_decrease():
    assert plain.starts([-3, 5, 2, 40, 7], 10).tolist() == [0, 5, 5, 10, 10]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("offsets", [None, [0, 3, 3, 9]])
def test_balance_gradient(score, offsets):
    rng = np.random.default_rng(3)
    T, E = 10, 6
    z = rng.normal(size=(T, E))
    z[4, 2] = -np.inf
    ids = rng.integers(-1, E, (T, 2))
    live = rng.random(T) < 0.8
    args = (ids, score, 0.7, 0.3, offsets, live)
    got = plain.balance(z, *args)
    finite = np.where(np.isinf(z), -60.0, z)
    want = differences(lambda z: plain.balance(z, *args)[0], finite)
    close(want, got[2])
    given = plain.balance(z, None, *args[1:], counts=got[1])
    assert given[0] == got[0] and np.array_equal(given[2], got[2])


def test_balance_by_hand():
    # even scores: the loss is its weight, whatever the counts
    loss, counts, dz = plain.balance(np.zeros((3, 4)), [[0, 1], [0, 2], [0, -1]], balance=0.5)
    assert loss == pytest.approx(0.5) and counts.tolist() == [[3, 1, 1, 0]]
    # a_e = 0.5 * 4 * c_e / 5 / 3, their mean 1/6 at each token
    assert np.allclose(dz[0], 0.25 * (0.5 * 4 / 15 * np.array([3, 1, 1, 0]) - 0.5 / 3))
    loss, _, dz = plain.balance(np.zeros((3, 4)), [[0, 1], [0, 2], [0, -1]], balance=0.0, z=1.0)
    assert loss == pytest.approx(np.log(4) ** 2)
    assert np.allclose(dz, 2 * np.log(4) / 4 / 3)
