"""Rules on logits and picking the next token on the GPU against the plain
implementation.

Adjusted logits are single binary32 operations, so they are equal bit for bit
(also after the one rounding to the output's type), and so are picked ids.
The logprob's softmax sum is made of float32 terms: with y = (top - z) / t, a
term is off by (2 y + 4) 2^-24 of its value, and a sum of at most 64 float32
additions deep by 64 * 2^-24; the mean of y under the softmax is at most
log V < 16, so the logarithm of the sum is off by at most
(32 + 4 + 64) 2^-24 < 7e-6; the value itself is rounded once to float32."""
import math
import threading

import numpy as np
import pytest

from gpu_util import device, note
from oracle import selection as plain

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SUM_ERROR = 100 * 2.0 ** -24


def lib():
    import greedy_iou_nms_amd as g
    return g


def to_gpu(a):
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int64) if a.dtype == np.uint64 else a).to(device())


def make_rules(rng, B, V, L=20, bias=5, masks=2, everything=True):
    """Rules as numpy arrays: repeated tokens, tokens outside the vocabulary,
    empty and full histories, unused and repeated bias entries."""
    u = {}
    if L:
        few = rng.integers(0, V, size=max(1, min(V, L // 2 + 1)))
        u["history"] = rng.choice(few, size=(B, L)).astype(np.int32)
        outside = rng.random((B, L)) < 0.1
        u["history"][outside] = rng.choice([-1, V, 2 ** 31 - 1, -2 ** 31], size=outside.sum())
        u["history_len"] = rng.integers(0, L + 1, size=B).astype(np.int32)
        u["history_len"][0] = L
        if B > 1:
            u["history_len"][1] = 0
        u["prompt_len"] = (u["history_len"] * rng.random(B)).astype(np.int32)
    if everything:
        u["repetition"] = rng.choice([1.0, 1.1, 0.9, 2.0], size=B).astype(np.float32)
        u["presence"] = rng.choice([0.0, 0.3, -0.3], size=B).astype(np.float32)
        u["frequency"] = rng.choice([0.0, 0.17, -0.1], size=B).astype(np.float32)
    if bias:
        u["bias_ids"] = rng.integers(-1, V + 1, size=(B, bias)).astype(np.int32)
        u["bias_values"] = (rng.normal(size=(B, bias)) * 3).astype(np.float32)
        u["bias_ids"][0, -1] = u["bias_ids"][0, 0]
    if masks:
        words = (V + 63) // 64
        u["allowed"] = rng.integers(-2 ** 63, 2 ** 63 - 1, size=(masks, words), dtype=np.int64)
        u["allowed_rows"] = rng.integers(-1, masks, size=B).astype(np.int32)
    return u


def gpu_rules(V, u):
    return lib().LogitRules(V, **{k: to_gpu(v) for k, v in u.items()})


def make_logits(rng, B, V, dtype, spread=3.0):
    z = torch.from_numpy(rng.normal(size=(B, V)) * spread).to(DTYPES[dtype])
    return z, z.float().numpy()


def same(got, want_f32):
    """Bit for bit in got's type, NaN for NaN."""
    want = torch.from_numpy(want_f32).to(got.dtype)
    got = got.cpu()
    ok = (got == want) | (torch.isnan(got) & torch.isnan(want))
    assert bool(ok.all()), int((~ok).sum())


def check_pick(z, adjusted, label="", rules=None, **kw):
    note("pick %s %s %s" % (label, tuple(z.shape),
                            {k: v if np.isscalar(v) else "." for k, v in kw.items()}))
    B = z.shape[0]
    kw.setdefault("max_top_k", 64)
    want_ids, want_lp = plain.pick(adjusted, kw["uniform"], kw["max_top_k"],
                                   *(kw.get(n) for n in ("temperature", "top_k", "top_p",
                                                         "min_p")))
    on = {k: to_gpu(v) if isinstance(v, np.ndarray) else v for k, v in kw.items()}
    ids, lp = lib().pick_tokens(z if z.is_cuda else z.to(device()), on.pop("uniform"),
                                rules=rules, **on)
    assert ids.shape == (B,) and ids.dtype == torch.int32 and lp.dtype == torch.float32
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    got = lp.cpu().numpy().astype(np.float64)
    inf = np.isinf(want_lp)
    np.testing.assert_array_equal(got[inf], want_lp[inf])
    tol = SUM_ERROR + 2.0 ** -24 * np.abs(want_lp[~inf])
    assert np.all(np.abs(got[~inf] - want_lp[~inf]) <= tol)
    return want_ids


def row_parameters(rng, B, k):
    return dict(uniform=rng.random(B).astype(np.float32),
                temperature=rng.choice([0.0, 0.5, 1.0, 1.7], size=B).astype(np.float32),
                top_k=rng.integers(0, k + 2, size=B).astype(np.int32),
                top_p=rng.choice([0.0, 0.3, 0.9, 1.0], size=B).astype(np.float32),
                min_p=rng.choice([0.0, 0.0, 0.1, 1.0], size=B).astype(np.float32), max_top_k=k)


# ------------------------------------------------------------------- adjust

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,V,L", [(1, 1, 1), (2, 2, 3), (3, 63, 10), (3, 64, 50), (2, 65, 1),
                                   (5, 1000, 200), (2, 8191, 333), (2, 16384, 2000),
                                   (3, 16385, 70), (2, 40001, 5000), (1, 100003, 30),
                                   (5, 131073, 600), (40, 114700, 900), (300, 17, 4097)])
def test_adjust_sizes(B, V, L, dtype):
    rng = np.random.default_rng([B, V, L])
    note("adjust %d %d %d %s" % (B, V, L, dtype))
    u = make_rules(rng, B, V, L)
    z, zf = make_logits(rng, B, V, dtype)
    same(lib().adjust_logits(z.to(device()), gpu_rules(V, u)), plain.adjust(zf, **u))


@pytest.mark.parametrize("leave_out", [
    ("prompt_len",), ("repetition",), ("presence",), ("frequency",),
    ("bias_ids", "bias_values"), ("allowed", "allowed_rows"),
    ("history", "history_len", "prompt_len"),
    ("history", "history_len", "prompt_len", "bias_ids", "bias_values"),
    ("history", "history_len", "prompt_len", "bias_ids", "bias_values", "allowed",
     "allowed_rows", "repetition", "presence", "frequency")])
def test_adjust_without(leave_out):
    rng = np.random.default_rng(1)
    u = {k: v for k, v in make_rules(rng, 4, 300).items() if k not in leave_out}
    z, zf = make_logits(rng, 4, 300, "f32")
    same(lib().adjust_logits(z.to(device()), gpu_rules(300, u)), plain.adjust(zf, **u))


def test_adjust_masks_by_row_number_and_outside():
    rng = np.random.default_rng(7)
    V = 130
    z, zf = make_logits(rng, 4, V, "f32")
    u = make_rules(rng, 4, V, masks=4)
    del u["allowed_rows"]
    same(lib().adjust_logits(z.to(device()), gpu_rules(V, u)), plain.adjust(zf, **u))
    u["allowed"][2] = 0
    u["allowed_rows"] = np.array([2, 4, -2 ** 31, 2 ** 31 - 1], np.int32)
    out = lib().adjust_logits(z.to(device()), gpu_rules(V, u))
    same(out, plain.adjust(zf, **u))
    assert bool(torch.isinf(out[[0, 1, 3]]).all())


def test_adjust_infinities_nan_and_lowest():
    rng = np.random.default_rng(8)
    for dtype in DTYPES:
        z, _ = make_logits(rng, 6, 500, dtype)
        lowest = torch.finfo(DTYPES[dtype]).min
        for row, v in enumerate((math.nan, math.inf, -math.inf, lowest, -lowest, 0.0)):
            z[row, ::3] = v
        z[5, 1::3] = -0.0
        u = make_rules(rng, 6, 500, L=400)
        zf = z.float().numpy()
        want = plain.adjust(zf, **u)
        got = lib().adjust_logits(z.to(device()), gpu_rules(500, u))
        same(got, want)
        assert bool((torch.isneginf(got.cpu().float()) | (torch.from_numpy(want) > -math.inf) |
                     torch.isnan(torch.from_numpy(want))).all())


def test_adjust_lengths_outside_the_capacity():
    rng = np.random.default_rng(9)
    u = make_rules(rng, 4, 50, L=30)
    u["history_len"] = np.array([31, 2 ** 31 - 1, -1, 30], np.int32)
    u["prompt_len"] = np.array([-5, 10, 3, 2 ** 31 - 1], np.int32)
    z, zf = make_logits(rng, 4, 50, "f32")
    same(lib().adjust_logits(z.to(device()), gpu_rules(50, u)), plain.adjust(zf, **u))
    u = make_rules(rng, 4, 50, L=30)
    u["history"] = u["history"][:, :0]
    u["history_len"] = u["prompt_len"] = np.full(4, 7, np.int32)
    same(lib().adjust_logits(z.to(device()), gpu_rules(50, u)), plain.adjust(zf, **u))


def test_adjust_in_place_strided_and_guarded():
    rng = np.random.default_rng(10)
    dev = device()
    B, V = 3, 1001
    u = make_rules(rng, B, V, L=100)
    for dtype in DTYPES:
        z, zf = make_logits(rng, B, V, dtype)
        want = plain.adjust(zf, **u)
        for shift in (0, 1, 3):
            wide = torch.full((B, V + 40), 9.0, dtype=DTYPES[dtype], device=dev)
            view = wide[:, shift:shift + V]
            view.copy_(z)
            # rules in rows of wider buffers
            r = {k: to_gpu(v) for k, v in u.items()}
            for name in ("history", "bias_ids", "bias_values", "allowed"):
                w = torch.zeros(r[name].shape[0], r[name].shape[1] + 5, dtype=r[name].dtype,
                                device=dev)
                w[:, 2:-3] = r[name]
                r[name] = w[:, 2:-3]
            rules = lib().LogitRules(V, **r)
            other = torch.full((B, V + 9), 9.0, dtype=DTYPES[dtype], device=dev)
            lib().adjust_logits(view, rules, out=other[:, 4:4 + V])
            same(other[:, 4:4 + V], want)
            assert bool((other[:, :4] == 9).all()) and bool((other[:, 4 + V:] == 9).all())
            assert lib().adjust_logits(view, rules, out=view) is view
            same(view, want)
            assert bool((wide[:, :shift] == 9).all()) and bool((wide[:, shift + V:] == 9).all())


def test_adjust_long_history_counts():
    # one token a hundred thousand times, beyond 16 bits
    dev = device()
    L, V = 100003, 700
    history = torch.full((2, L), 5, dtype=torch.int32, device=dev)
    history[1, ::2] = 699
    length = torch.tensor([L, L - 1], dtype=torch.int32, device=dev)
    rules = lib().LogitRules(V, history=history, history_len=length,
                             frequency=torch.full((2,), 2.0 ** -10, device=dev))
    out = lib().adjust_logits(torch.zeros(2, V, device=dev), rules).cpu()
    assert out[0, 5] == -L / 1024 and out[1, 5] == -50001 / 1024 and out[1, 699] == -50001 / 1024
    assert int((out != 0).sum()) == 3


# --------------------------------------------------------------------- pick

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,V,k", [(1, 1, 1), (2, 2, 2), (3, 63, 5), (3, 64, 64), (2, 65, 100),
                                   (4, 1000, 1), (4, 1000, 17), (3, 4097, 200), (2, 16384, 50),
                                   (3, 16385, 1024), (2, 40001, 300), (1, 100003, 64),
                                   (1, 100003, 1024), (2, 262147, 40)])
def test_pick_sizes(B, V, k, dtype):
    rng = np.random.default_rng([B, V, k])
    z, zf = make_logits(rng, B, V, dtype)
    for _ in range(3):
        check_pick(z, zf, **row_parameters(rng, B, k))
    u = make_rules(rng, B, V, L=min(V, 300))
    check_pick(z, plain.adjust(zf, **u), "rules", rules=gpu_rules(V, u),
               **row_parameters(rng, B, k))


@pytest.mark.parametrize("k", [1, 2, 63, 64, 65, 255, 256, 257, 1000, 1024])
def test_pick_all_of_the_candidates(k):
    """Every rank is drawn once: the order of all k candidates is checked."""
    rng = np.random.default_rng(k)
    V = 5000
    z = (rng.integers(-2000, 2000, size=(1, V)) / 512).astype(np.float32)
    order = np.argsort(-z[0].astype(np.float64), kind="stable")[:k]
    w = np.exp(z[0, order].astype(np.float64) - z[0].max())
    cum = np.cumsum(w)
    u = ((cum - w / 2) / cum[-1]).astype(np.float32)
    ids = check_pick(torch.from_numpy(z.repeat(k, 0)), z.repeat(k, 0), uniform=u, max_top_k=k)
    # the middle of each candidate's share: every rank, in order
    assert (ids == order).mean() > 0.99


@pytest.mark.parametrize("V", [5, 300, 20000, 70000])
@pytest.mark.parametrize("k", [1, 3, 64, 700])
def test_pick_ties(V, k):
    rng = np.random.default_rng([V, k])
    z = np.zeros((6, V), np.float32)
    z[1] = rng.integers(0, 2, size=V)
    z[2] = rng.integers(0, 5, size=V) / 4
    z[3, V // 2:] = 1.0
    z[4, ::2] = -0.0                # equal to +0
    z[5, -1] = 1.0
    for _ in range(2):
        check_pick(torch.from_numpy(z), z, uniform=rng.random(6).astype(np.float32), max_top_k=k)


@pytest.mark.parametrize("V", [40, 1000, 50000])
@pytest.mark.parametrize("order", [1, -1])
def test_pick_sorted_rows(V, order):
    """The largest values all in one place: the first or the last tokens."""
    rng = np.random.default_rng(V)
    z = (np.arange(V)[::order] / 64 % 4096).astype(np.float32)[None].repeat(2, 0)
    for k in (1, 30, 900):
        check_pick(torch.from_numpy(z), z, uniform=rng.random(2).astype(np.float32), max_top_k=k)


@pytest.mark.parametrize("V", [64, 1000, 33000])
@pytest.mark.parametrize("k", [1, 20, 500])
def test_pick_masked_and_infinite(V, k):
    rng = np.random.default_rng([V, k])
    z = rng.normal(size=(9, V)).astype(np.float32)
    z[0] = -np.inf
    z[1] = np.nan
    z[2, 1:] = -np.inf
    z[3, ::2] = np.nan
    z[4, 7] = np.inf
    z[5, ::5] = np.inf
    z[6] = np.finfo(np.float32).min
    z[7, : V - 3] = np.finfo(np.float32).min
    u = rng.random(9).astype(np.float32)
    check_pick(torch.from_numpy(z), z, uniform=u, max_top_k=k)
    # a mask that leaves nothing, one token, a whole word, all
    words = (V + 63) // 64
    allowed = np.zeros((3, words), np.int64)
    allowed[1, (V - 1) // 64] = np.int64(1) << ((V - 1) % 64 if (V - 1) % 64 < 63 else 62)
    allowed[2, 0] = -1
    rules = dict(allowed=allowed, allowed_rows=np.array([0, 1, 2, 0, 1, 2, 9, 2, 1], np.int32))
    check_pick(torch.from_numpy(z), plain.adjust(z, **rules), "masks", uniform=u, max_top_k=k,
               rules=gpu_rules(V, rules))


def test_pick_extreme_parameters():
    rng = np.random.default_rng(12)
    z, zf = make_logits(rng, 8, 900, "f32")
    nan, inf = math.nan, math.inf
    below_one = np.nextafter(np.float32(1), np.float32(0))
    base = row_parameters(rng, 8, 30)
    base["temperature"][:] = 1.0

    def with_(**kw):
        return {**base, **{k: np.array(v, base[k].dtype) for k, v in kw.items()}}

    check_pick(z, zf, **with_(uniform=[0.0, below_one] * 4))
    check_pick(z, zf, **with_(top_k=[0, -1, 1, 30, 31, 2 ** 31 - 1, -2 ** 31, 2]))
    check_pick(z, zf, **with_(temperature=[1e-30, 1e30, 1e-6, 50.0, 0.01, 1e-38, 3e38, 0.1]))
    check_pick(z, zf, **with_(top_p=[-1.0, 0.0, 2.0, inf, -inf, 1e-30, below_one, 0.5]))
    check_pick(z, zf, **with_(min_p=[-1.0, 2.0, inf, -inf, 1.0, 1e-30, below_one, 0.5]))
    # what is not a number takes the first token
    dev = device()
    first = torch.from_numpy(zf.argmax(axis=1).astype(np.int32))
    for name in ("uniform", "temperature", "top_p", "min_p"):
        kw = {k: to_gpu(v) if isinstance(v, np.ndarray) else v for k, v in base.items()}
        kw[name] = torch.full((8,), nan, device=dev)
        ids, lp = lib().pick_tokens(z.to(dev), **kw)
        assert torch.equal(ids.cpu(), first) and bool(torch.isfinite(lp).all())


def test_pick_strided_and_offset_rows():
    rng = np.random.default_rng(13)
    for dtype in DTYPES:
        z, zf = make_logits(rng, 4, 3000, dtype)
        wide = torch.full((8, 3037), 50.0, dtype=DTYPES[dtype], device=device())
        for shift in (0, 1, 2, 5, 37):
            wide.fill_(50.0)
            view = wide[::2, shift:shift + 3000]
            view.copy_(z)
            check_pick(view, zf, **row_parameters(rng, 4, 20))
        one = wide[2:3, 37:]
        check_pick(one, zf[1:2], **row_parameters(rng, 1, 20))


@pytest.mark.parametrize("V", [700, 9000, 30000, 70000])
@pytest.mark.parametrize("k", [1, 2, 50, 1000])
def test_pick_crowded_rows(V, k):
    """More equal or neighbouring values at the bound than there is room for."""
    rng = np.random.default_rng([V, k])
    z = rng.normal(size=(12, V)).astype(np.float32)
    low = np.finfo(np.float32).min
    z[0] = 0.0
    z[1] = low
    z[2, 40:] = low
    z[3, :V - 40] = low
    z[4] = np.round(z[4] * 2) / 2
    z[5] = -np.sort(-z[5])
    z[6] = np.sort(z[6])
    z[7] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    z[8] = np.float32(2.0) ** rng.integers(-140, 120, size=V).astype(np.float32)
    z[9] = np.inf
    z[9, ::2] = -np.inf
    z[10] = 1.0 + np.float32(2.0 ** -23) * rng.integers(0, 3, size=V).astype(np.float32)
    z[11, ::5] = z[11].max()
    check_pick(torch.from_numpy(z), z, uniform=rng.random(12).astype(np.float32), max_top_k=k,
               temperature=np.full(12, 2.0, np.float32))
    u = rng.random(12).astype(np.float32)
    check_pick(torch.from_numpy(z).half(), torch.from_numpy(z).half().float().numpy(), uniform=u,
               max_top_k=k)


def test_rows_more_than_2_to_31_elements_apart():
    rng = np.random.default_rng(16)
    stride, V = 2 ** 31 + 40, 33000
    flat = torch.empty(2 * stride + V, dtype=torch.bfloat16, device=device())
    apart = flat.as_strided((3, V), (stride, 1))
    z, zf = make_logits(rng, 3, V, "bf16")
    u = make_rules(rng, 3, V, L=30)
    apart.copy_(z)
    check_pick(apart, plain.adjust(zf, **u), rules=gpu_rules(V, u), **row_parameters(rng, 3, 20))
    assert lib().adjust_logits(apart, gpu_rules(V, u), out=apart) is apart
    same(apart, plain.adjust(zf, **u))


def test_pick_many_rows():
    rng = np.random.default_rng(14)
    z, zf = make_logits(rng, 700, 700, "bf16")
    u = make_rules(rng, 700, 700, L=50)
    check_pick(z, plain.adjust(zf, **u), rules=gpu_rules(700, u), **row_parameters(rng, 700, 12))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,V,k", [(70, 65537, 1), (70, 65537, 33), (52, 81921, 700),
                                   (257, 20000, 20), (40, 40000, 1000), (3, 140001, 1)])
def test_pick_rows_of_several_slices(B, V, k, dtype):
    rng = np.random.default_rng([B, V, k])
    z, zf = make_logits(rng, B, V, dtype)
    u = make_rules(rng, B, V, L=800)
    check_pick(z, plain.adjust(zf, **u), rules=gpu_rules(V, u), **row_parameters(rng, B, k))


@pytest.mark.parametrize("B,V", [(2, 30000), (2, 90000), (70, 65537)])
@pytest.mark.parametrize("k", [1, 50, 900])
def test_pick_outliers_and_crowds(B, V, k):
    """A few values far above, crowds of equal ones, and masks by the lowest
    value of the type, whose distance no bin resolves."""
    rng = np.random.default_rng([B, V, k])
    z = rng.normal(size=(B, V)).astype(np.float32)
    z[0, ::7] = 1.25
    z[0, 5] = 3e38
    z[1] = np.finfo(np.float32).min
    z[1, rng.integers(0, V, size=k // 2 + 1)] = 1.0
    z[1, V - 1] = 1e30
    for b in range(2, B):
        z[b, rng.random(V) < 0.99] = np.finfo(np.float32).min
    check_pick(torch.from_numpy(z), z, uniform=rng.random(B).astype(np.float32), max_top_k=k)


@pytest.mark.parametrize("V,k", [(30, 5), (9000, 40), (70000, 900), (70000, 1)])
def test_infinite_temperature_draws_evenly(V, k):
    rng = np.random.default_rng(V)
    z, zf = make_logits(rng, 4, V, "f16")
    z[1, ::3] = -math.inf
    zf = z.float().numpy()
    check_pick(z, zf, uniform=rng.random(4).astype(np.float32), max_top_k=k,
               temperature=np.full(4, np.inf, np.float32))


def test_a_table_without_masks():
    rng = np.random.default_rng(17)
    z, zf = make_logits(rng, 3, 500, "f32")
    u = dict(allowed=np.zeros((0, 8), np.int64), allowed_rows=np.array([-1, 0, 3], np.int32))
    want = plain.adjust(zf, **u)
    assert np.isfinite(want[0]).all() and np.isinf(want[1:]).all()
    same(lib().adjust_logits(z.to(device()), gpu_rules(500, u)), want)
    check_pick(z, want, rules=gpu_rules(500, u), **row_parameters(rng, 3, 9))


def test_pick_no_rows():
    dev = device()
    ids, lp = lib().pick_tokens(torch.zeros(0, 10, device=dev), torch.zeros(0, device=dev))
    assert ids.shape == (0,) and lp.shape == (0,)
    z = torch.zeros(0, 10, device=dev)
    assert lib().adjust_logits(z, lib().LogitRules(10)).shape == (0, 10)


# ------------------------------------------------------------- used together

class Loop:
    """A decode loop: routed experts' outputs make the hidden state, logits
    come from it, a token is picked under the rules and joins the history."""

    def __init__(self, dev, B=5, V=2000, D=32, E=16, k=3, L=12):
        rng = np.random.default_rng(20)
        self.B, self.V, self.k = B, V, k

        def t(*shape):
            return torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(dev)

        self.embed, self.router, self.experts = t(V, D), t(D, E), t(E, D)
        self.head, self.bias = t(D, V) * 0.3, t(E) * 0.1
        self.history = torch.zeros(B, L, dtype=torch.int32, device=dev)
        self.length = torch.ones(B, dtype=torch.int32, device=dev)
        self.prompt = torch.ones(B, dtype=torch.int32, device=dev)
        self.uniform = torch.zeros(B, device=dev)
        self.allowed = torch.from_numpy(rng.integers(-2 ** 63, 2 ** 63 - 1, size=(3, (V + 63) // 64),
                                                     dtype=np.int64)).to(dev)
        self.allowed_rows = torch.tensor([0, 1, -1, 2, -1][:B], dtype=torch.int32, device=dev)
        self.fields = dict(history=self.history, history_len=self.length, prompt_len=self.prompt,
                           repetition=torch.full((B,), 1.3, device=dev),
                           frequency=torch.full((B,), 0.2, device=dev), allowed=self.allowed,
                           allowed_rows=self.allowed_rows)
        self.rules = lib().LogitRules(V, **self.fields)
        self.temperature = torch.tensor([0.0, 1.0, 0.7, 1.0, 1.5][:B], device=dev)

    def start(self, first):
        self.history.zero_()
        self.history[:, 0] = first
        self.length.fill_(1)

    def step(self):
        last = self.history.gather(1, self.length.long()[:, None] - 1)[:, 0]
        h = self.embed[last.long()]
        scores = (h[:, :, None] * self.router[None]).sum(1)
        experts, weights = lib().route_experts(scores, self.k, score="sigmoid", bias=self.bias)
        h = h + (self.experts[experts.long()] * weights[:, :, None]).sum(1)
        logits = (h[:, :, None] * self.head[None]).sum(1)
        ids, logprobs = lib().pick_tokens(logits, self.uniform, max_top_k=20,
                                          temperature=self.temperature, rules=self.rules)
        adjusted = lib().adjust_logits(logits, self.rules)
        self.history.scatter_(1, self.length.long()[:, None], ids[:, None])
        self.length.add_(1)
        return scores, experts, weights, logits, adjusted, ids, logprobs

    def expected(self, scores, logits, history, length):
        want_e, want_w, _ = plain.route(scores.cpu().numpy(), self.k, "sigmoid",
                                        self.bias.cpu().numpy())
        u = {k: v.cpu().numpy() for k, v in self.fields.items()}
        u.update(history=history, history_len=length)
        adjusted = plain.adjust(logits.cpu().numpy(), **u)
        ids, lp = plain.pick(adjusted, self.uniform.cpu().numpy(), 20,
                             self.temperature.cpu().numpy())
        return want_e, want_w, adjusted, ids, lp


def test_decode_loop_eager_and_captured():
    dev = device()
    loop = Loop(dev)
    first = torch.arange(1, 6, dtype=torch.int32, device=dev)
    draws = torch.rand(8, 5, generator=torch.Generator().manual_seed(3)).to(dev)
    loop.start(first)
    tokens = []
    for s in range(8):
        loop.uniform.copy_(draws[s])
        history, length = loop.history.cpu().numpy(), loop.length.cpu().numpy()
        scores, experts, weights, logits, adjusted, ids, lp = loop.step()
        want = loop.expected(scores, logits, history, length)
        np.testing.assert_array_equal(experts.cpu().numpy(), want[0])
        np.testing.assert_allclose(weights.cpu().numpy(), want[1], rtol=2.0 ** -21)
        np.testing.assert_array_equal(adjusted.cpu().numpy(), want[2])
        np.testing.assert_array_equal(ids.cpu().numpy(), want[3])
        np.testing.assert_allclose(lp.cpu().numpy(), want[4], rtol=2.0 ** -24, atol=SUM_ERROR)
        tokens.append(ids.cpu())
    # captured once, replayed for every step, with eager steps of another loop
    # and waits between the replays
    loop.start(first)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loop.step()
    torch.cuda.current_stream().wait_stream(side)
    loop.start(first)
    with torch.cuda.graph(graph):
        out = loop.step()
    loop.start(first)
    other = Loop(dev, B=3, V=333)
    other.start(first[:3])
    for s in range(8):
        loop.uniform.copy_(draws[s])
        graph.replay()
        other.step()
        torch.cuda.synchronize()
        assert torch.equal(out[5].cpu(), tokens[s])


def test_two_captured_graphs_at_the_same_time():
    dev = device()
    rng = np.random.default_rng(21)
    z = [torch.from_numpy(rng.normal(size=(4, 50000)).astype(np.float32) * 3).to(dev)
         for _ in range(2)]
    u = [torch.full((4,), 0.3, device=dev), torch.full((4,), 0.8, device=dev)]
    want = [lib().pick_tokens(z[i], u[i], max_top_k=200) for i in range(2)]
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(lib().pick_tokens(z[i], u[i], max_top_k=200))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                for t in outs[i]:
                    t.zero_()
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])


def test_two_streams_at_the_same_time():
    dev = device()
    rng = np.random.default_rng(22)
    V = 30000
    z, zf = make_logits(rng, 3, V, "f32")
    z = z.to(dev)
    kw = [row_parameters(rng, 3, 60) for _ in range(2)]
    want = [plain.pick(zf, k["uniform"], 60, k["temperature"], k["top_k"], k["top_p"],
                       k["min_p"])[0] for k in kw]
    on = [{n: to_gpu(v) if isinstance(v, np.ndarray) else v for n, v in k.items()} for k in kw]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(lib().pick_tokens(z, **on[i])[0])
    torch.cuda.synchronize()
    for i in range(2):
        for ids in got[i]:
            np.testing.assert_array_equal(ids.cpu().numpy(), want[i])


def test_threads_at_the_same_time():
    """Each thread has a stream of its own; calls of different sizes."""
    dev = device()
    rng = np.random.default_rng(24)
    work = []
    for B, V, k in ((3, 40000, 700), (7, 900, 4), (2, 70000, 1), (30, 20000, 60)):
        z, zf = make_logits(rng, B, V, "f32")
        u = make_rules(rng, B, V, L=100)
        kw = row_parameters(rng, B, k)
        want, _ = plain.pick(plain.adjust(zf, **u), kw["uniform"], k, kw["temperature"],
                             kw["top_k"], kw["top_p"], kw["min_p"])
        on = {n: to_gpu(v) if isinstance(v, np.ndarray) else v for n, v in kw.items()}
        work.append((z.to(dev), gpu_rules(V, u), on, want))
    torch.cuda.synchronize()
    wrong = []

    def run(first):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = []
            for i in range(20):
                z, rules, on, want = work[(first + i) % len(work)]
                got.append((lib().pick_tokens(z, rules=rules, **on)[0], want))
            torch.cuda.current_stream().synchronize()
            wrong.extend(first for ids, want in got if not np.array_equal(ids.cpu().numpy(), want))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []


def test_results_do_not_depend_on_the_run():
    dev = device()
    rng = np.random.default_rng(23)
    V = 70001
    z, _ = make_logits(rng, 6, V, "bf16")
    u = make_rules(rng, 6, V, L=3000)
    rules = gpu_rules(V, u)
    z = z.to(dev)
    uniform = to_gpu(rng.random(6).astype(np.float32))
    first = lib().pick_tokens(z, uniform, max_top_k=500, rules=rules)
    for _ in range(10):
        again = lib().pick_tokens(z, uniform, max_top_k=500, rules=rules)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_refusals():
    dev = device()
    g = lib()
    z = torch.zeros(4, 100, device=dev)
    u = torch.zeros(4, device=dev)
    for k in (0, -1, 1025):
        with pytest.raises(g.NMSError) as e:
            g.pick_tokens(z, u, max_top_k=k)
        assert e.value.status == "NMS_INVALID_ARG"
    with pytest.raises(ValueError):
        g.pick_tokens(z, u, max_top_k=2 ** 32 + 5)
    with pytest.raises(TypeError):
        g.pick_tokens(z, u, rules={"repetition": u})
    with pytest.raises(TypeError):
        g.adjust_logits(z, None)
    with pytest.raises(TypeError):
        g.pick_tokens(z, None)
    with pytest.raises(ValueError):
        g.pick_tokens(z, u[:3])
    with pytest.raises(ValueError):
        g.pick_tokens(z, u.cpu())
    with pytest.raises(TypeError):
        g.pick_tokens(z, u, top_k=u)
    with pytest.raises(ValueError):
        g.pick_tokens(z, u, rules=g.LogitRules(99))
    with pytest.raises(ValueError):
        g.pick_tokens(z, u, rules=g.LogitRules(100, repetition=u[:3]))
    with pytest.raises(TypeError):
        g.adjust_logits(z, g.LogitRules(100), out=z.half())
    with pytest.raises(ValueError):
        g.adjust_logits(z, g.LogitRules(100), out=torch.zeros(4, 101, device=dev))
    with pytest.raises(ValueError):
        g.adjust_logits(z.t(), g.LogitRules(4))
    with pytest.raises(ValueError):
        g.LogitRules(100, history=torch.zeros(4, 5, dtype=torch.int32, device=dev))
    with pytest.raises(ValueError):
        g.LogitRules(100, repetition=u, presence=u[:2])
    with pytest.raises(g.NMSError) as e:
        g.adjust_logits(z, g.LogitRules(100, bias_ids=torch.zeros(4, 2048, dtype=torch.int32,
                                                                  device=dev),
                                        bias_values=torch.zeros(4, 2048, device=dev)))
    assert e.value.status == "NMS_TOO_LARGE"
