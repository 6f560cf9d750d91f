"""Refusals of the losses that need no GPU: the C entry points' host checks and
the binding's checks of tensors."""
import ctypes

import pytest
import torch

import greedy_iou_nms_amd as g
from greedy_iou_nms_amd import losses as mod

FAKE = 0x10000      # never dereferenced: every call below fails its host checks
BIG = 1 << 40
lib = g._lib
NAN, INF = float("nan"), float("inf")


def name(status):
    return g._STATUS[status]


def size(rows, vocab, pairs=0):
    out = ctypes.c_size_t(7)
    return name(lib.nms_loss_workspace_size(rows, vocab, pairs, ctypes.byref(out))), out.value


def test_workspace_sizes():
    assert size(4, 100)[0] == "NMS_OK" and size(4, 100)[1] >= 64
    assert size(0, 1)[0] == "NMS_OK"
    assert size(-1, 100) == ("NMS_INVALID_ARG", 0)
    assert size(1, 0) == ("NMS_INVALID_ARG", 0)
    assert size(1, 1, -1) == ("NMS_INVALID_ARG", 0)
    assert size(65537, 100) == ("NMS_TOO_LARGE", 0)
    assert size(1, (1 << 22) + 1) == ("NMS_TOO_LARGE", 0)
    assert size(1, 1, 32769) == ("NMS_TOO_LARGE", 0)
    assert name(lib.nms_loss_workspace_size(1, 1, 0, None)) == "NMS_INVALID_ARG"
    # monotone in the rows where slices are, so that a kept workspace serves smaller calls
    assert size(65536, 1 << 22)[1] >= 65536 * 24

    def balance(tokens, experts, sequences, top_k):
        out = ctypes.c_size_t(7)
        return name(lib.nms_balance_workspace_size(tokens, experts, sequences, top_k,
                                                   ctypes.byref(out)))
    assert balance(10, 4, 1, 2) == "NMS_OK" and balance(0, 1, 1, 0) == "NMS_OK"
    for bad in ((-1, 4, 1, 2), (1, 0, 1, 2), (1, 4, 0, 2), (1, 4, 1, -1), (1, 4, 1, 65)):
        assert balance(*bad) == "NMS_INVALID_ARG", bad
    for bad in ((1 << 25, 4, 1, 2), (1, 1025, 1, 2), (1, 4, 65537, 2)):
        assert balance(*bad) == "NMS_TOO_LARGE", bad


ROWS = dict(logits=FAKE, dtype=0, rows=4, vocab=100, stride=100, tokens=FAKE)
SPACE = dict(ws=FAKE, ws_bytes=BIG)


def logprobs(logprobs=FAKE, **kw):
    r = {**ROWS, **SPACE, **kw}
    return name(lib.nms_token_logprobs(r["logits"], r["dtype"], r["rows"], r["vocab"],
                                       r["stride"], r["tokens"], None, logprobs, None, r["ws"],
                                       r["ws_bytes"], None))


def backward(g=FAKE, out=FAKE, out_stride=100, **kw):
    r = {**ROWS, **SPACE, **kw}
    return name(lib.nms_token_logprobs_backward(
        r["logits"], r["dtype"], r["rows"], r["vocab"], r["stride"], r["tokens"], None, g, None,
        out, out_stride, r["ws"], r["ws_bytes"], None))


def policy(options=(0.2, 0.2, 0.0, 0.0), old=FAKE, adv=FAKE, ref=None, loss=FAKE, out=FAKE,
           out_stride=100, **kw):
    r = {**ROWS, **SPACE, **kw}
    o = None if options is None else ctypes.byref(mod._PolicyOptions(*options))
    return name(lib.nms_policy_loss(
        r["logits"], r["dtype"], r["rows"], r["vocab"], r["stride"], r["tokens"], old, adv, None,
        ref, None, o, None, loss, None, None, out, out_stride, r["ws"], r["ws_bytes"], None))


def preference(options=(0, 0, 0.1, 0.0, 0.0), offsets=FAKE, pairs=2, loss=FAKE, lp=FAKE,
               margins=FAKE, out=FAKE, out_stride=100, back=False, **kw):
    r = {**ROWS, **SPACE, **kw}
    o = None if options is None else ctypes.byref(mod._PreferenceOptions(*options))
    head = (r["logits"], r["dtype"], r["rows"], r["vocab"], r["stride"], r["tokens"], offsets,
            pairs)
    if back:
        return name(lib.nms_preference_loss_backward(*head, None, o, margins, None, out,
                                                     out_stride, r["ws"], r["ws_bytes"], None))
    return name(lib.nms_preference_loss(*head, None, None, o, None, loss, lp, margins, out,
                                        out_stride, r["ws"], r["ws_bytes"], None))


CALLS = [logprobs, backward, policy, preference,
         lambda **kw: preference(back=True, **kw)]


@pytest.mark.parametrize("call", CALLS)
def test_rows_of_logits(call):
    for bad in (dict(logits=None), dict(logits=FAKE + 2), dict(logits=FAKE + 1, dtype=2),
                dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(vocab=0), dict(stride=99),
                dict(tokens=None), dict(ws=None), dict(ws=FAKE + 128)):
        assert call(**bad) == "NMS_INVALID_ARG", bad
    assert call(rows=65537) == "NMS_TOO_LARGE"
    assert call(vocab=(1 << 22) + 1, stride=1 << 23) == "NMS_TOO_LARGE"
    assert call(ws_bytes=0) == "NMS_WORKSPACE_TOO_SMALL"


@pytest.mark.parametrize("call", CALLS[1:])
def test_gradients_of_rows(call):
    for bad in (dict(out=FAKE + 1), dict(out_stride=99)):
        assert call(**bad) == "NMS_INVALID_ARG", bad


def test_token_logprobs_arguments():
    assert logprobs(logprobs=None) == "NMS_INVALID_ARG"
    assert logprobs(rows=0, logits=None, tokens=None, logprobs=None, ws=None) == "NMS_OK"
    assert backward(g=None) == "NMS_INVALID_ARG"
    assert backward(out=None) == "NMS_INVALID_ARG"
    assert backward(rows=0, logits=None, tokens=None, g=None, out=None, ws=None) == "NMS_OK"


def test_policy_arguments():
    for bad in ((-0.1, 0.2, 0, 0), (1.1, 0.2, 0, 0), (NAN, 0.2, 0, 0), (0.2, -0.1, 0, 0),
                (0.2, INF, 0, 0), (0.2, NAN, 0, 0), (0.2, 0.2, -1, 0), (0.2, 0.2, NAN, 0),
                (0.2, 0.2, INF, 0), (0.2, 0.2, 0, NAN), (0.2, 0.2, 0, INF), None):
        assert policy(bad, ref=FAKE) == "NMS_INVALID_ARG", bad
    assert policy((0.2, 0.2, 0.1, 0)) == "NMS_INVALID_ARG"  # no reference
    assert policy(old=None) == "NMS_INVALID_ARG"
    assert policy(adv=None) == "NMS_INVALID_ARG"
    assert policy(loss=None, out=None) == "NMS_INVALID_ARG"


def test_preference_arguments():
    for back in (False, True):
        for bad in ((3, 0, 0.1, 0, 0), (-1, 0, 0.1, 0, 0), (0, 0, 0.0, 0, 0), (0, 0, -1, 0, 0),
                    (0, 0, NAN, 0, 0), (0, 0, INF, 0, 0), (0, 0, 0.1, -0.1, 0),
                    (0, 0, 0.1, 0.6, 0), (0, 0, 0.1, NAN, 0), (1, 0, 0.1, 0.1, 0),
                    (2, 0, 0.1, 0.1, 0), (0, 0, 0.1, 0, NAN), (0, 0, 0.1, 0, INF), None):
            assert preference(bad, back=back) == "NMS_INVALID_ARG", bad
        assert preference(pairs=0, back=back) == "NMS_INVALID_ARG"
        assert preference(pairs=32769, back=back) == "NMS_TOO_LARGE"
        assert preference(offsets=None, back=back) == "NMS_INVALID_ARG"
        assert preference(offsets=FAKE + 4, back=back) == "NMS_INVALID_ARG"
        assert preference(margins=None, back=back) == "NMS_INVALID_ARG"
    assert preference(loss=None) == "NMS_INVALID_ARG"
    assert preference(lp=None) == "NMS_INVALID_ARG"
    assert preference(out=None, back=True) == "NMS_INVALID_ARG"


def balance(options=(0, 2, 1.0, 0.0), logits=FAKE, dtype=0, tokens=4, experts=8, stride=8,
            ids=FAKE, offsets=None, sequences=1, loss=FAKE, counts=FAKE, out=FAKE, out_stride=8,
            ws=FAKE, ws_bytes=BIG):
    o = None if options is None else ctypes.byref(mod._BalanceOptions(*options))
    return name(lib.nms_balance_loss(logits, dtype, tokens, experts, stride, ids, None, offsets,
                                     sequences, o, None, loss, counts, out, out_stride, ws,
                                     ws_bytes, None))


def test_balance_arguments():
    for bad in ((2, 2, 1, 0), (-1, 2, 1, 0), (0, -1, 1, 0), (0, 65, 1, 0), (0, 2, NAN, 0),
                (0, 2, INF, 0), (0, 2, 1, NAN), (0, 2, 1, INF), None):
        assert balance(bad) == "NMS_INVALID_ARG", bad
    for bad in (dict(logits=None), dict(logits=FAKE + 2), dict(dtype=3), dict(tokens=-1),
                dict(experts=0), dict(stride=7), dict(ids=None, counts=None),
                dict(sequences=0), dict(sequences=2), dict(offsets=FAKE + 4),
                dict(out_stride=7), dict(out=FAKE + 2), dict(ws=None), dict(ws=FAKE + 8),
                dict(loss=None, counts=None, out=None)):
        assert balance(**bad) == "NMS_INVALID_ARG", bad
    assert balance(experts=1025, stride=1025, out_stride=1025) == "NMS_TOO_LARGE"
    assert balance(tokens=(1 << 24) + 1) == "NMS_TOO_LARGE"
    assert balance(offsets=FAKE, sequences=65537) == "NMS_TOO_LARGE"
    assert balance(ws_bytes=64) == "NMS_WORKSPACE_TOO_SMALL"


def test_balance_without_ids_or_counts():
    """Where ids are NULL the counts are read, so that one of the two has to be
    there, for an empty batch and for tokens without a place too."""
    none = dict(ids=None, counts=None)
    assert balance((0, 0, 1.0, 0.0), **none) == "NMS_INVALID_ARG"
    assert balance((0, 0, 1.0, 0.0), tokens=9000, **none) == "NMS_INVALID_ARG"
    assert balance((0, 0, 1.0, 0.0), offsets=FAKE, sequences=3, **none) == "NMS_INVALID_ARG"
    for top_k in (0, 2):
        o = (0, top_k, 1.0, 0.0)
        assert balance(o, tokens=0, **none) == "NMS_INVALID_ARG"
        assert balance(o, tokens=0, logits=None, out=None, **none) == "NMS_INVALID_ARG"
        assert balance(o, tokens=0, loss=None, **none) == "NMS_INVALID_ARG"
        assert balance(o, tokens=0, offsets=FAKE, sequences=3, **none) == "NMS_INVALID_ARG"


# ------------------------------------------------------------------ the binding

class Claimed(torch.Tensor):
    is_cuda = True


def on_gpu(*shape, dtype=torch.float32, **kw):
    return torch.zeros(*shape, dtype=dtype, **kw).as_subclass(Claimed)


I32, I64 = torch.int32, torch.int64


def tokens(n=4):
    return on_gpu(n, dtype=I32)


def test_binding_refuses_tensors():
    z, f = on_gpu(4, 9), on_gpu(4)
    calls = {
        "logprobs": lambda z=z, a=tokens(), t=None: g.token_logprobs(z, a, t),
        "backward": lambda z=z, a=tokens(), t=None: g.token_logprobs_backward(z, a, f, t),
        "policy": lambda z=z, a=tokens(), t=None: g.policy_loss(z, a, f, f, temperature=t),
        "both": lambda z=z, a=tokens(), t=None: g.policy_loss_with_grad(z, a, f, f,
                                                                        temperature=t),
    }
    for call in calls.values():
        with pytest.raises(TypeError):
            call(a=None)
        with pytest.raises(TypeError):
            call(a=on_gpu(4, dtype=I64))
        with pytest.raises(ValueError):
            call(a=tokens(3))
        with pytest.raises(ValueError):
            call(a=on_gpu(8, dtype=I32)[::2])
        with pytest.raises(TypeError):
            call(t=on_gpu(4, dtype=torch.float64))
        with pytest.raises(ValueError):
            call(t=on_gpu(5))
        with pytest.raises(TypeError):
            call(z=on_gpu(4, 9, dtype=torch.float64))
        with pytest.raises(ValueError):
            call(z=on_gpu(4, 9, 1))
        with pytest.raises(ValueError):
            call(z=on_gpu(9, 4).t())
        with pytest.raises(ValueError):
            call(z=torch.zeros(4, 9))
        with pytest.raises(TypeError):
            call(z=None)
    with pytest.raises(TypeError):
        g.policy_loss(z, tokens(), None, f)
    with pytest.raises(TypeError):
        g.policy_loss(z, tokens(), f, None)
    with pytest.raises(ValueError):
        g.policy_loss(z, tokens(), f, f, on_gpu(3))
    with pytest.raises(TypeError):
        g.policy_loss_with_grad(z, tokens(), f, f, grad_loss=2.0)
    with pytest.raises(TypeError):
        g.policy_loss_with_grad(z, tokens(), f, f, grad_loss=on_gpu(1, dtype=torch.float16))
    with pytest.raises(ValueError):
        g.policy_loss_with_grad(z, tokens(), f, f, grad_loss=on_gpu(2))
    at = on_gpu(3, dtype=I64)
    for bad in (on_gpu(2, dtype=I64), on_gpu(4, dtype=I64), on_gpu(1, dtype=I64),
                on_gpu(3, 1, dtype=I64)):
        with pytest.raises(ValueError):
            g.preference_loss(z, tokens(), bad)
    with pytest.raises(TypeError):
        g.preference_loss(z, tokens(), [0, 2, 4])
    with pytest.raises(TypeError):
        g.preference_loss(z, tokens(), on_gpu(3, dtype=I32))
    with pytest.raises(TypeError):
        g.preference_loss(z, None, at)
    with pytest.raises(ValueError):
        g.preference_loss(z, tokens(), at, ref_logprobs=on_gpu(1))
    with pytest.raises(ValueError):
        g.preference_loss(z, tokens(), at, weights=on_gpu(2))


def test_binding_refuses_balance_tensors():
    z, ids = on_gpu(4, 9), on_gpu(4, 2, dtype=I32)
    for bad in (dict(ids=None), dict(ids=on_gpu(4, dtype=I32)), dict(ids=on_gpu(3, 2, dtype=I32)),
                dict(ids=on_gpu(4, 4, dtype=I32)[:, ::2]), dict(counts=on_gpu(9, dtype=I32)),
                dict(ids=None, counts=on_gpu(8, dtype=I32)), dict(ids=None, counts=on_gpu(9)),
                dict(offsets=on_gpu(1, dtype=I64)), dict(live=on_gpu(3, dtype=torch.bool)),
                dict(ids=None, counts=on_gpu(9, dtype=I32), offsets=on_gpu(3, dtype=I64)),
                dict(grad_loss=on_gpu(0))):
        with pytest.raises(ValueError):
            g.balance_loss_with_grad(z, **{"ids": ids, **bad})
    for bad in (dict(ids=on_gpu(4, 2, dtype=I64)), dict(offsets=on_gpu(2, dtype=I32)),
                dict(offsets=[0, 4]), dict(live=on_gpu(4)), dict(ids=None, counts=[1] * 9)):
        with pytest.raises(TypeError):
            g.balance_loss_with_grad(z, **{"ids": ids, **bad})


def test_tensors_that_require_a_gradient():
    """What a loss has no gradient in is refused where it requires one."""
    z, a, f = on_gpu(4, 9), tokens(), on_gpu(4)
    leaf = on_gpu(4).requires_grad_()
    with pytest.raises(RuntimeError, match="temperature"):
        g.token_logprobs(z, a, leaf)
    for at in range(5):
        given = [f, f, f, f, f]
        given[at] = leaf
        with pytest.raises(RuntimeError, match="has no gradient in"):
            g.policy_loss(z, a, *given)
    at = on_gpu(3, dtype=I64)
    with pytest.raises(RuntimeError, match="ref_logprobs"):
        g.preference_loss(z, a, at, ref_logprobs=on_gpu(2).requires_grad_())
    with pytest.raises(RuntimeError, match="weights"):
        g.preference_loss(z, a, at, weights=on_gpu(1).requires_grad_())


def test_options_that_are_refused():
    z, a, f = on_gpu(4, 9), tokens(), on_gpu(4)
    with pytest.raises(ValueError, match="kind"):
        mod._preference_options("logistic", False, 0.1, 0.0, 0.0)
    with pytest.raises(ValueError, match="score"):
        mod._balance_options("tanh", 2, 1.0, 0.0)
