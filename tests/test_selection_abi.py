"""Refusals of the selection operators that need no GPU: the C entry points'
host checks and the binding's checks of tensors."""
import ctypes

import pytest
import torch

import greedy_iou_nms_amd as g
from greedy_iou_nms_amd import selection as sel

FAKE = 0x10000      # never dereferenced: every call below fails its host checks
lib = g._lib


def name(status):
    return g._STATUS[status]


def options(score=0, top_k=2, renormalise=1, scale=1.0, groups=1, kept=1, top=1):
    return sel._RouteOptions(score, top_k, renormalise, scale, groups, kept, top)


def route(o=None, logits=FAKE, dtype=0, tokens=4, experts=8, stride=8, ids=FAKE, weights=FAKE,
          null=False):
    o = options() if o is None else o
    return name(lib.nms_route_experts(logits, dtype, tokens, experts, stride, None, None,
                                      None if null else ctypes.byref(o), ids, weights, None, None))


def route_back(o=None, logits=FAKE, dtype=0, tokens=4, experts=8, stride=8, ids=FAKE, gw=FAKE,
               out=FAKE, out_stride=8):
    o = options() if o is None else o
    return name(lib.nms_route_experts_backward(logits, dtype, tokens, experts, stride, ids, gw,
                                               ctypes.byref(o), out, out_stride, None))


def test_route_arguments():
    for bad in (options(score=2), options(top_k=0), options(top_k=65), options(top_k=9),
                options(scale=float("nan")), options(scale=float("inf")), options(groups=0),
                options(groups=3), options(groups=2, kept=0), options(groups=2, kept=3),
                options(groups=4, kept=1, top_k=3), options(top=0), options(top=3)):
        assert route(bad) == "NMS_INVALID_ARG"
    assert route(null=True) == "NMS_INVALID_ARG"
    assert route(logits=None) == "NMS_INVALID_ARG"
    assert route(logits=FAKE + 2) == "NMS_INVALID_ARG"
    assert route(logits=FAKE + 1, dtype=2) == "NMS_INVALID_ARG"
    assert route(dtype=3) == "NMS_INVALID_ARG"
    assert route(tokens=-1) == "NMS_INVALID_ARG"
    assert route(experts=0) == "NMS_INVALID_ARG"
    assert route(stride=7) == "NMS_INVALID_ARG"
    assert route(ids=None) == "NMS_INVALID_ARG"
    assert route(weights=None) == "NMS_INVALID_ARG"
    assert route(experts=1025, stride=1025) == "NMS_TOO_LARGE"
    assert route(tokens=(1 << 30) + 1) == "NMS_TOO_LARGE"


def test_route_backward_arguments():
    for bad in (options(score=-1), options(top_k=0), options(top_k=65),
                options(scale=float("nan"))):
        assert route_back(bad) == "NMS_INVALID_ARG"
    assert route_back(ids=None) == "NMS_INVALID_ARG"
    assert route_back(gw=None) == "NMS_INVALID_ARG"
    assert route_back(out=None) == "NMS_INVALID_ARG"
    assert route_back(out_stride=7) == "NMS_INVALID_ARG"
    assert route_back(stride=0) == "NMS_INVALID_ARG"
    assert route_back(experts=1025, stride=1025, out_stride=1025) == "NMS_TOO_LARGE"
    assert route_back(tokens=0, logits=None, out=None) == "NMS_OK"


def rules(**kw):
    return sel._LogitRules(**kw)


def adjust(u=None, logits=FAKE, dtype=0, rows=2, vocab=100, stride=100, out=FAKE, out_stride=100,
           null=False):
    u = rules() if u is None else u
    return name(lib.nms_adjust_logits(logits, dtype, rows, vocab, stride,
                                      None if null else ctypes.byref(u), out, out_stride, None))


BAD_RULES = [
    dict(history=FAKE, history_stride=4, history_capacity=4),
    dict(history=FAKE, history_len=FAKE, history_stride=3, history_capacity=4),
    dict(history=FAKE, history_len=FAKE, history_stride=4, history_capacity=-1),
    dict(history_len=FAKE),
    dict(prompt_len=FAKE),
    dict(bias_count=-1),
    dict(bias_count=2, bias_stride=2, bias_ids=FAKE),
    dict(bias_count=2, bias_stride=2, bias_values=FAKE),
    dict(bias_count=2, bias_stride=1, bias_ids=FAKE, bias_values=FAKE),
    dict(allowed=FAKE, allowed_stride=1, allowed_count=1),
    dict(allowed=FAKE, allowed_stride=2, allowed_count=-1),
    dict(allowed=FAKE + 4, allowed_stride=2, allowed_count=2),
    dict(allowed_rows=FAKE),
]


def test_adjust_arguments():
    for bad in BAD_RULES:
        assert adjust(rules(**bad)) == "NMS_INVALID_ARG", bad
    assert adjust(rules(history=FAKE, history_len=FAKE, history_stride=1 << 20,
                        history_capacity=1 << 20)) == "NMS_TOO_LARGE"
    assert adjust(rules(bias_count=2048, bias_stride=2048, bias_ids=FAKE,
                        bias_values=FAKE)) == "NMS_TOO_LARGE"
    assert adjust(null=True) == "NMS_INVALID_ARG"
    assert adjust(logits=None) == "NMS_INVALID_ARG"
    assert adjust(out=None) == "NMS_INVALID_ARG"
    assert adjust(stride=99) == "NMS_INVALID_ARG"
    assert adjust(out_stride=99) == "NMS_INVALID_ARG"
    assert adjust(dtype=-1) == "NMS_INVALID_ARG"
    assert adjust(rows=-1) == "NMS_INVALID_ARG"
    assert adjust(vocab=0) == "NMS_INVALID_ARG"
    assert adjust(rows=65537) == "NMS_TOO_LARGE"
    assert adjust(vocab=(1 << 22) + 1, stride=1 << 23, out_stride=1 << 23) == "NMS_TOO_LARGE"
    assert adjust(rows=0, logits=None, out=None) == "NMS_OK"


def pick(u=None, logits=FAKE, dtype=0, rows=2, vocab=100, stride=100, uniform=FAKE, max_top_k=5,
         ids=FAKE, logprobs=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return name(lib.nms_pick_tokens(logits, dtype, rows, vocab, stride,
                                    None if u is None else ctypes.byref(u), uniform, None, None,
                                    None, None, max_top_k, ids, logprobs, ws, ws_bytes, None))


def test_pick_arguments():
    for bad in BAD_RULES:
        assert pick(rules(**bad)) == "NMS_INVALID_ARG", bad
    assert pick(uniform=None) == "NMS_INVALID_ARG"
    assert pick(ids=None) == "NMS_INVALID_ARG"
    assert pick(logprobs=None) == "NMS_INVALID_ARG"
    assert pick(ws=None) == "NMS_INVALID_ARG"
    assert pick(ws=FAKE + 128) == "NMS_INVALID_ARG"
    assert pick(max_top_k=0) == "NMS_INVALID_ARG"
    assert pick(max_top_k=1025) == "NMS_INVALID_ARG"
    assert pick(logits=None) == "NMS_INVALID_ARG"
    assert pick(stride=99) == "NMS_INVALID_ARG"
    assert pick(rows=65537) == "NMS_TOO_LARGE"
    assert pick(rows=0, logits=None, ws=None) == "NMS_OK"
    need = g.pick_workspace_size(2, 100, 5)
    assert pick(ws_bytes=need - 1) == "NMS_WORKSPACE_TOO_SMALL"


def test_pick_workspace_size():
    out = ctypes.c_size_t(7)
    assert name(lib.nms_pick_workspace_size(1, 100, 5, None)) == "NMS_INVALID_ARG"
    assert name(lib.nms_pick_workspace_size(1, 0, 5, ctypes.byref(out))) == "NMS_INVALID_ARG"
    assert name(lib.nms_pick_workspace_size(1, 100, 0, ctypes.byref(out))) == "NMS_INVALID_ARG"
    assert name(lib.nms_pick_workspace_size(65537, 9, 5, ctypes.byref(out))) == "NMS_TOO_LARGE"
    assert out.value == 0
    # it grows with every size, and stays near the candidates' 8 bytes for
    # each of max_top_k per 1024 tokens of a row
    assert g.pick_workspace_size(4, 200000, 64) >= g.pick_workspace_size(2, 200000, 64)
    assert g.pick_workspace_size(4, 200000, 64) <= 4 * (200000 // 1024 + 1) * (64 * 8 + 64) + 4096


def test_binding_refuses_unusable_tensors():
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        g.route_experts(cpu, 2)                                # not on a GPU
    with pytest.raises(TypeError):
        g.route_experts([[0.0]], 1)
    with pytest.raises(ValueError):
        g.adjust_logits(cpu, g.LogitRules(8))
    with pytest.raises(ValueError):
        g.pick_tokens(cpu, torch.zeros(4))
    with pytest.raises(ValueError):
        g.LogitRules(8, repetition=torch.ones(4))              # not on a GPU
    with pytest.raises(TypeError):
        g.LogitRules(8, repetition=1.1)
    # the checks themselves need no GPU
    dev = cpu.device
    assert sel._rows(cpu, "x", dev) == 8
    assert sel._rows(torch.zeros(4, 16)[:, :8], "x", dev) == 16
    assert sel._rows(torch.zeros(1, 8).expand(1, 8), "x", dev) == 8
    for bad in (torch.zeros(8, 4).t(), torch.zeros(1, 8).expand(4, 8), torch.zeros(8),
                torch.zeros(4, 16)[:, ::2]):
        with pytest.raises(ValueError):
            sel._rows(bad, "x", dev)
    with pytest.raises(TypeError):
        sel._rows(cpu.double(), "x", dev)
    with pytest.raises(ValueError):
        sel._rows(cpu, "x", dev, torch.Size((4, 9)))
    with pytest.raises(ValueError):
        sel._rows(cpu, "x", torch.device("meta"))
    assert sel._vector(None, "x", 4, torch.float32, dev) is None
    with pytest.raises(TypeError):
        sel._vector(torch.zeros(4, dtype=torch.int64), "x", 4, torch.int32, dev)
    with pytest.raises(ValueError):
        sel._vector(torch.zeros(5), "x", 4, torch.float32, dev)
    with pytest.raises(ValueError):
        sel._vector(torch.zeros(8)[::2], "x", 4, torch.float32, dev)
    with pytest.raises(ValueError):
        sel._route_options("relu", 2, True, 1.0, 1, None, 2)


def test_rules_have_to_fit_each_other(monkeypatch):
    """LogitRules' checks, with tensors that only claim to be on a GPU."""
    class Claimed(torch.Tensor):
        is_cuda = True

    def t(*shape, dtype=torch.int32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(Claimed)

    def f(*shape):
        return t(*shape, dtype=torch.float32)

    good = dict(history=t(3, 5), history_len=t(3), prompt_len=t(3), repetition=f(3),
                bias_ids=t(3, 2), bias_values=f(3, 2), allowed=t(4, 2, dtype=torch.int64),
                allowed_rows=t(3))
    r = g.LogitRules(100, **good)
    assert r.rows == 3 and r._struct.history_capacity == 5 and r._struct.allowed_count == 4
    r._for(3, 100, torch.device("cpu"))
    for args in ((4, 100, torch.device("cpu")), (3, 99, torch.device("cpu")),
                 (3, 100, torch.device("meta"))):
        with pytest.raises(ValueError):
            r._for(*args)
    for change in (dict(history=None), dict(history_len=None), dict(bias_ids=None),
                   dict(bias_values=None), dict(allowed=None), dict(history_len=t(2)),
                   dict(bias_values=f(3, 3)), dict(allowed=t(4, 1, dtype=torch.int64)),
                   dict(allowed_rows=None), dict(repetition=f(3, 1)),
                   dict(bias_ids=t(3, 4)[:, :2])):
        with pytest.raises(ValueError):
            g.LogitRules(100, **{**good, **change})
    for change in (dict(history=f(3, 5)), dict(repetition=t(3)),
                   dict(allowed=t(4, 2)), dict(history_len=t(3, dtype=torch.int64))):
        with pytest.raises(TypeError):
            g.LogitRules(100, **{**good, **change})
