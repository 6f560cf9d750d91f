"""The balance loss of routing on the GPU against the plain 64-bit one."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gpu_util import device, note  # noqa: E402
from loss_util import SMALL, TYPES, U, dev, host, lib, logits_of, within  # noqa: E402
from oracle import losses as plain  # noqa: E402

pytestmark = pytest.mark.gpu


def bounds(z, dtype, want, f, score, balance, zc, S, n_tokens, up):
    """Loss and gradient of a row may be off by their terms times the number of
    their roundings: an exponential has 4 x + 2 of them (x the distance to the
    row's largest, or to 0 for a sigmoid), sums over E experts E / 8 + 16, the
    rest 16; lse = m + log s is off by those of s and 2 U of itself."""
    E = z.shape[1]
    fin = np.where(np.isfinite(z), z, 0.0)
    top = np.where(np.isfinite(z), z, -np.inf).max(axis=1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    x = np.where(np.isfinite(z), top - z, 0.0)
    far = np.minimum(np.maximum(x, np.abs(fin)), 200.0)
    p = np.where(np.isfinite(z), np.exp(-x), 0.0)
    p /= np.maximum(p.sum(axis=1, keepdims=True), 1e-300)
    s = p
    if score == "sigmoid":
        logs = np.where(np.isfinite(z), -np.logaddexp(0, -fin), -np.inf)
        hi = logs.max(axis=1, keepdims=True)
        s = np.exp(logs - np.where(np.isfinite(hi), hi, 0.0))
        s /= np.maximum(s.sum(axis=1, keepdims=True), 1e-300)
    mean = (s * far).sum(axis=1, keepdims=True) + (p * far).sum(axis=1, keepdims=True)
    rel = U * (4 * far + 4 * mean + E / 4 + 48)
    inner = (f * s).sum(axis=1, keepdims=True)
    lse = top + np.log(np.maximum(np.exp(np.where(np.isfinite(z), -x, -np.inf)).sum(
        axis=1, keepdims=True), 1e-300))
    per = zc / max(1, n_tokens)
    err_lse = rel.max(axis=1, keepdims=True) + 2 * U * np.abs(lse)
    grad = abs(up) * (rel * s * (f + inner) * 2 + 2 * per * p * (np.abs(lse) * rel * 2 + err_lse))
    loss = (rel.max(axis=1) * inner[:, 0] * 2 + per * 3 * (np.abs(lse) * err_lse)[:, 0]).sum()
    half = torch.finfo(dtype).eps / 2
    return loss, grad * (1 + half) + half * np.abs(want) + SMALL[dtype]


def factors(z, counts, at, live, balance):
    T, E = z.shape
    f = np.zeros((T, E))
    S = len(at) - 1
    for q in range(S):
        mine = np.arange(at[q], at[q + 1])
        mine = mine[live[mine]]
        if len(mine) and counts[q].sum():
            f[mine] = balance / S * E * counts[q] / counts[q].sum() / len(mine)
    return f


CASES = [(1, 1, 1, 1), (3, 2, 1, 1), (7, 4, 2, 1), (100, 8, 2, 3), (65, 60, 4, 1),
         (1001, 64, 6, 1), (300, 65, 3, 5), (257, 128, 8, 2), (70, 200, 8, 70), (513, 256, 8, 7),
         (90, 300, 5, 1), (33, 512, 8, 2), (40, 777, 4, 1), (20, 1024, 12, 3), (9000, 16, 8, 1),
         (40000, 5, 2, 1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k,S", CASES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance(T, E, k, S, score, dtype):
    note("balance %d %d %d %d %s %s" % (T, E, k, S, score, dtype))
    rng = np.random.default_rng(T + E + k)
    z = logits_of(rng, T, E, dtype, 1.5, stride=E + 3 if T % 2 else None)
    if E > 4:
        z[torch.from_numpy(rng.random((T, E)) < 0.05).to(device())] = -float("inf")
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    ids[rng.random((T, k)) < 0.01] = E + 5
    live = rng.random(T) < 0.85
    offsets = None
    if S > 1:
        offsets = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int64)
        offsets[1] = offsets[2] if S > 2 else offsets[1]
    up, balance, zc = 64.0, 0.7, 0.2
    for weight in (0.0, zc):
        loss, counts, dz = plain.balance(host(z), ids, score, balance, weight, offsets, live,
                                         up=up)
        at = np.array([0, T]) if offsets is None else plain.starts(offsets, T)
        f = factors(host(z), counts, at, live, balance)
        used = np.zeros(T, bool)
        used[at[0]:at[-1]] = live[at[0]:at[-1]]
        zz = np.where(used[:, None], host(z), -np.inf)
        err, tol = bounds(zz, dtype, dz, f, score, balance, weight, S, used.sum(), up)
        given = dict(score=score, balance=balance, z=weight, offsets=dev(offsets),
                     live=dev(live))
        got = lib().balance_loss(z, dev(ids), **given)
        shaped = counts if S > 1 else counts[0]
        assert np.array_equal(got[1].cpu().numpy(), shaped)
        within(host(got[0]), loss, err + 2 * U * abs(loss), "loss")
        both = lib().balance_loss_with_grad(z, dev(ids), grad_loss=dev(np.float32([up])), **given)
        assert np.array_equal(both[2].cpu().numpy(), shaped)
        assert torch.equal(both[0], got[0])
        within(host(both[1]), dz, tol, "gradient")
        # by counts that are given, and through autograd
        by = lib().balance_loss_with_grad(z, counts=got[1], grad_loss=dev(np.float32([up])),
                                          **given)
        assert torch.equal(by[0], got[0]) and torch.equal(by[1], both[1])
        leaf = z.clone().requires_grad_()
        loss2, counts2 = lib().balance_loss(leaf, dev(ids), **given)
        loss2.backward(torch.tensor(up, device=device()))
        assert torch.equal(loss2.detach(), got[0]) and torch.equal(leaf.grad, both[1])
        # in place of the logits
        there = z.clone()
        lib().balance_loss_with_grad(there, dev(ids), grad_loss=dev(np.float32([up])),
                                     out=there, **given)
        assert torch.equal(there, both[1])


def test_balance_of_long_sequences():
    """Sequences whose ids are counted in parts, against counts by torch."""
    note("balance long")
    rng = np.random.default_rng(4)
    T, E, k = 60001, 7, 8
    z = logits_of(rng, T, E, torch.float32)
    ids = dev(rng.integers(-1, E, (T, k)).astype(np.int32))
    live = dev(rng.random(T) < 0.9)
    offsets = np.array([3, 30000, 30000, 59990], np.int64)
    loss, counts = lib().balance_loss(z, ids, offsets=dev(offsets), live=live)
    for q in range(3):
        own = ids[offsets[q]:offsets[q + 1]][live[offsets[q]:offsets[q + 1]]]
        want = torch.bincount((own.reshape(-1) + 1).long(), minlength=E + 1)[1:]
        assert torch.equal(counts[q].long(), want)
    again = lib().balance_loss(z, counts=counts, offsets=dev(offsets), live=live)
    assert torch.equal(loss, again[0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", TYPES)
def test_balance_odd_values(score, dtype):
    """Rows without an expert, rows of the lowest value, far below 0 and above;
    NaN shows, but not in padded rows."""
    note("balance odd %s %s" % (score, dtype))
    rng = np.random.default_rng(6)
    z = logits_of(rng, 8, 12, dtype)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    z[0] = -float("inf")
    z[1] = low
    z[2, 1:] = low
    z[3] -= 300.0
    z[4] += 300.0
    z[5] = high
    z[6] = float("nan")
    z[7, 3:] = -float("inf")
    ids = rng.integers(0, 12, (8, 2)).astype(np.int32)
    live = np.arange(8) != 6
    loss, counts, dz = plain.balance(host(z), ids, score, 0.5, 0.0, None, live)
    f = factors(host(z), counts, [0, 8], live, 0.5)
    zz = np.where(live[:, None], host(z), -np.inf)
    err, tol = bounds(zz, dtype, dz, f, score, 0.5, 0.0, 1, 7, 1.0)
    got = lib().balance_loss_with_grad(z, dev(ids), score=score, balance=0.5, live=dev(live))
    within(host(got[0]), loss, err + 2 * U * abs(loss), "loss")
    within(host(got[1]), dz, tol, "gradient")
    loss, dz, _ = lib().balance_loss_with_grad(z, dev(ids), score=score, balance=0.5)
    assert np.isnan(host(loss)) and np.isnan(host(dz)[6]).all()
    assert np.isfinite(host(dz)[[0, 1, 2, 3, 4, 5, 7]]).all()


def test_balance_without_tokens_or_places():
    z = torch.zeros(6, 4, device=device())
    ids = torch.zeros(6, 2, dtype=torch.int32, device=device())
    loss, dz, counts = lib().balance_loss_with_grad(
        z, ids, z=1.0, live=torch.zeros(6, dtype=torch.bool, device=device()))
    assert float(loss) == 0 and not host(dz).any() and counts.tolist() == [0] * 4
    loss, dz, counts = lib().balance_loss_with_grad(z, ids[:, :0])
    assert float(loss) == 0 and not host(dz).any() and counts.tolist() == [0] * 4


def test_balance_beside_routing():
    """As a training step makes them: experts and their weights, the balance loss
    of the same logits, one gradient."""
    note("balance beside routing")
    rng = np.random.default_rng(10)
    g = lib()
    z = logits_of(rng, 120, 32, torch.float32)
    live = dev(rng.random(120) < 0.9)
    factor = dev(rng.normal(size=(120, 4)).astype(np.float32))
    leaf = z.clone().requires_grad_()
    ids, w, counts = g.route_experts(leaf, 4, "sigmoid", live=live, counts=True)
    loss, counted = g.balance_loss(leaf, ids, "sigmoid", balance=0.01, z=0.001, live=live)
    assert torch.equal(counts, counted)
    ((w * factor).sum() + loss).backward()
    a = g.route_experts_backward(z, ids, factor, "sigmoid")
    b = g.balance_loss_with_grad(z, ids, "sigmoid", balance=0.01, z=0.001, live=live)[1]
    assert torch.equal(leaf.grad, a + b) or torch.equal(leaf.grad, b + a)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [(40, 12, None), (5000, 60, None), (900, 33, [0, 1, 500, 890])])
def test_balance_by_given_counts_through_autograd(size, score):
    """Counts that are given go through autograd as ids do: the factors come from
    the same counts, so that loss and gradient have the same bits; the counts
    themselves stay as they are, and take no gradient."""
    note("balance by counts %s %s" % (size, score))
    T, E, offsets = size
    rng = np.random.default_rng(12)
    z = logits_of(rng, T, E, torch.float32)
    ids = dev(rng.integers(-1, E, (T, 3)).astype(np.int32))
    given = dict(score=score, balance=0.3, z=0.01, live=dev(rng.random(T) < 0.9),
                 offsets=None if offsets is None else dev(np.array(offsets, np.int64)))
    up = dev(np.float32([1.5]))
    want = lib().balance_loss_with_grad(z, ids, grad_loss=up, **given)
    counts = want[2].clone()
    for _ in range(2):  # the same tensor twice
        leaf = z.clone().requires_grad_()
        loss, got = lib().balance_loss(leaf, counts=counts, **given)
        assert not got.requires_grad and not counts.requires_grad
        (loss * up[0]).backward()
        assert torch.equal(loss.detach(), want[0])
        assert torch.equal(leaf.grad, want[1])
        assert torch.equal(got, want[2]) and torch.equal(counts, want[2])
