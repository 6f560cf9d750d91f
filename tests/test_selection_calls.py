"""What the binding of the selection operators hands to the library, without a
GPU: the library's entry points are replaced by ones that note their arguments,
and the tensors only claim to be on a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import greedy_iou_nms_amd as g
from greedy_iou_nms_amd import selection as sel


class Claimed(torch.Tensor):
    is_cuda = True


def on_gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Claimed)


class Library:
    """Notes the arguments of each call; the options as they are at the call."""

    def __init__(self):
        self.calls = []

    def _note(self, name, args):
        self.calls.append((name, args))
        return 0

    def nms_route_experts(self, *args):
        o = ctypes.cast(args[7], ctypes.POINTER(sel._RouteOptions)).contents
        return self._note("route", dict(top_k=o.top_k, scale=o.scale, groups=o.groups,
                                        kept_groups=o.kept_groups, renormalise=o.renormalise))

    def nms_route_experts_backward(self, *args):
        o = ctypes.cast(args[7], ctypes.POINTER(sel._RouteOptions)).contents
        return self._note("back", dict(top_k=o.top_k, scale=o.scale, renormalise=o.renormalise))

    def nms_pick_workspace_size(self, rows, vocab, k, out):
        ctypes.cast(out, ctypes.POINTER(ctypes.c_size_t)).contents.value = 8 * rows * k
        return self._note("size", (rows, vocab, k))

    def nms_pick_tokens(self, *args):
        return self._note("pick", args)

    def nms_adjust_logits(self, *args):
        return self._note("adjust", args)

    def last(self):
        return self.calls[-1][1]


@pytest.fixture
def library(monkeypatch):
    fake = Library()
    monkeypatch.setattr(sel, "_lib", fake)
    monkeypatch.setattr(sel, "_current_device", lambda: None)  # a CPU device's index
    monkeypatch.setattr(sel, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(sel, "_capturing", lambda: False)
    sel._pick_workspace_size.cache_clear()
    yield fake
    sel._pick_workspace_size.cache_clear()  # the sizes here are made up


# ------------------------------------------------- numbers, not their holders

def test_options_are_read_at_every_call(library):
    """A tensor's value may change between two calls with the same tensor."""
    z = on_gpu(4, 8)
    scale, k = torch.tensor(2.5), torch.tensor(3)
    for value, count in ((2.5, 3), (4.0, 5), (1.0, 2)):
        scale.fill_(value)
        k.fill_(count)
        ids, w = g.route_experts(z, k, scale=scale)
        assert library.last()["scale"] == value and library.last()["top_k"] == count
        assert ids.shape == (4, count) and w.shape == (4, count)
        g.route_experts_backward(z, on_gpu(4, 2, dtype=torch.int32), on_gpu(4, 2), scale=scale)
        assert library.last()["scale"] == value and library.last()["top_k"] == 2
    keep = torch.tensor(True)
    for value in (True, False):
        keep.fill_(value)
        g.route_experts(z, 2, renormalise=keep)
        assert library.last()["renormalise"] == int(value)


def test_whole_numbers_of_other_types(library):
    z = on_gpu(4, 8)
    g.route_experts(z, np.int64(3), groups=np.int32(2), kept_groups=np.int8(1))
    assert [library.last()[n] for n in ("top_k", "groups", "kept_groups")] == [3, 2, 1]


@pytest.mark.parametrize("name", ["top_k", "groups", "kept_groups", "group_top"])
def test_a_wrong_type_is_refused_after_a_right_one(library, name):
    """4.0 is no whole number, whatever was called before."""
    z = on_gpu(4, 8)
    kw = dict(top_k=2, groups=2, kept_groups=2, group_top=2)
    g.route_experts(z, **kw)
    with pytest.raises(TypeError):
        g.route_experts(z, **{**kw, name: 2.0})


def test_pick_sizes_are_read_at_every_call(library):
    k = torch.tensor(5)
    z, u = on_gpu(3, 100), on_gpu(3)
    for count in (5, 9):
        k.fill_(count)
        assert g.pick_workspace_size(3, 100, k) == 8 * 3 * count
        g.pick_tokens(z, u, max_top_k=k)
        assert library.last()[11] == count and library.last()[15] >= 8 * 3 * count
    for bad in ((3.0, 100, 5), (3, 100.0, 5), (3, 100, 5.0)):
        with pytest.raises(TypeError):
            g.pick_workspace_size(*bad)
    for bad in ((2 ** 64 + 3, 100, 5), (3, 2 ** 64 + 100, 5), (3, 100, 2 ** 32 + 5)):
        with pytest.raises(ValueError):
            g.pick_workspace_size(*bad)


# --------------------------------------------------------- where the rules are

def rules_of(library):
    """The struct that the last adjust call was given."""
    return library.last()[5]._obj


def test_rules_follow_a_history_that_grows(library):
    z = on_gpu(2, 100)
    history = on_gpu(2, 8, dtype=torch.int32)
    rules = g.LogitRules(100, history=history, history_len=on_gpu(2, dtype=torch.int32))
    g.adjust_logits(z, rules)
    before = history.data_ptr()
    assert rules_of(library).history == before and rules_of(library).history_capacity == 8
    history.resize_(2, 5000)
    assert history.data_ptr() != before
    g.adjust_logits(z, rules)
    assert rules_of(library).history == history.data_ptr()
    assert rules_of(library).history_capacity == rules_of(library).history_stride == 5000
    g.pick_tokens(z, on_gpu(2), rules=rules)
    assert library.last()[5]._obj.history == history.data_ptr()


def test_rules_follow_other_memory_and_other_shapes(library):
    z = on_gpu(2, 100)
    wide = on_gpu(2, 40, dtype=torch.int32)
    history, length = on_gpu(2, 8, dtype=torch.int32), on_gpu(2, dtype=torch.int32)
    values, allowed = on_gpu(2), on_gpu(2, 2, dtype=torch.int64)
    rules = g.LogitRules(100, history=history, history_len=length, repetition=values,
                         allowed=allowed)
    history.data = wide[:, 4:20]
    length.set_(on_gpu(2, dtype=torch.int32))
    values.data = on_gpu(2) + 1
    allowed.set_(on_gpu(2, 7, dtype=torch.int64))
    g.adjust_logits(z, rules)
    u = rules_of(library)
    assert (u.history, u.history_stride, u.history_capacity) == (wide.data_ptr() + 16, 40, 16)
    assert u.history_len == length.data_ptr() and u.repetition == values.data_ptr()
    assert u.allowed == allowed.data_ptr() and u.allowed_stride == 7
    # the same address, another shape
    at = history.data_ptr()
    history.set_(wide.untyped_storage(), 4, (2, 10), (20, 1))
    assert history.data_ptr() == at
    g.adjust_logits(z, rules)
    u = rules_of(library)
    assert (u.history, u.history_stride, u.history_capacity) == (at, 20, 10)


def test_rules_hold_the_memory_that_they_read(library):
    """Nothing else may be put where the struct points to."""
    values = on_gpu(3)
    rules = g.LogitRules(100, repetition=values)
    held = rules._memory[0].untyped_storage()._cdata
    assert held == values.untyped_storage()._cdata
    values.data = on_gpu(3)
    assert rules._memory[0].untyped_storage()._cdata == held
    assert rules._memory[0].data_ptr() == rules._struct.repetition != values.data_ptr()


def test_rules_that_no_longer_fit_are_refused(library):
    z = on_gpu(2, 100)

    def make():
        t = dict(history=on_gpu(2, 8, dtype=torch.int32),
                 history_len=on_gpu(2, dtype=torch.int32), repetition=on_gpu(2),
                 allowed=on_gpu(2, 2, dtype=torch.int64))
        return t, g.LogitRules(100, **t)

    for name, other, error in (("history", on_gpu(3, 8, dtype=torch.int32), ValueError),
                               ("repetition", on_gpu(3), ValueError),
                               ("allowed", on_gpu(2, 1, dtype=torch.int64), ValueError),
                               ("history", on_gpu(2, 16, dtype=torch.int32)[:, ::2],
                                ValueError)):
        t, rules = make()
        g.adjust_logits(z, rules)
        calls = len(library.calls)
        t[name].set_(other)
        for call in (lambda: g.adjust_logits(z, rules),
                     lambda: g.pick_tokens(z, on_gpu(2), rules=rules)):
            for _ in range(2):
                with pytest.raises(error):
                    call()
        assert len(library.calls) == calls


# ------------------------------------------------------------- an empty batch

def test_an_empty_batch_with_full_rules():
    """Tensors without rows have no address; the library itself is called."""
    lib = g._lib
    t = dict(history=on_gpu(0, 5, dtype=torch.int32), history_len=on_gpu(0, dtype=torch.int32),
             prompt_len=on_gpu(0, dtype=torch.int32), repetition=on_gpu(0), presence=on_gpu(0),
             frequency=on_gpu(0), bias_ids=on_gpu(0, 3, dtype=torch.int32),
             bias_values=on_gpu(0, 3), allowed=on_gpu(0, 2, dtype=torch.int64),
             allowed_rows=on_gpu(0, dtype=torch.int32))
    for leave_out in ((), ("allowed_rows",), ("history", "history_len", "prompt_len"),
                      ("bias_ids", "bias_values")):
        ref = g.LogitRules(100, **{k: v for k, v in t.items() if k not in leave_out})._ref
        assert lib.nms_adjust_logits(None, 0, 0, 100, 100, ref, None, 100, None) == 0
        assert lib.nms_pick_tokens(None, 0, 0, 100, 100, ref, None, None, None, None, None, 5,
                                   None, None, None, 0, None) == 0
    # what is wrong whatever the rows are is refused all the same
    many = g.LogitRules(100, bias_ids=on_gpu(0, 2048, dtype=torch.int32),
                        bias_values=on_gpu(0, 2048))
    assert g._STATUS[lib.nms_adjust_logits(None, 0, 0, 100, 100, many._ref, None, 100,
                                           None)] == "NMS_TOO_LARGE"


# ------------------------------------------------------------------ workspaces

def test_workspace_of_its_own(library):
    """NMS tells its own words in its workspace from older ones by a tag of 32
    bits; what picking leaves behind would be mistaken for them now and then."""
    nms_buf = g._default_workspace(torch.device("cpu"), 0).get(1 << 16, torch.device("cpu"))
    g.pick_tokens(on_gpu(3, 100), on_gpu(3))
    first = library.last()[14]
    assert not nms_buf.data_ptr() <= first < nms_buf.data_ptr() + nms_buf.numel()
    g.pick_tokens(on_gpu(2, 100), on_gpu(2))
    assert library.last()[14] == first                      # kept
    assert g._default_workspace(torch.device("cpu"), 0).buf is nms_buf


def test_a_call_to_be_refused_allocates_nothing(monkeypatch):
    """top_k above the limit, as far as an int goes: the library refuses it
    before any output of that width is made."""
    monkeypatch.setattr(sel, "_current_device", lambda: None)
    monkeypatch.setattr(sel, "_raw_stream", lambda device: 0)
    made = []
    empty = torch.empty

    def noted(*shape, **kw):
        made.append(shape)
        assert np.prod(shape[0] if isinstance(shape[0], tuple) else shape) < 1 << 20
        return empty(*shape, **kw)

    monkeypatch.setattr(sel.torch, "empty", noted)
    for k in (0, -1, -2 ** 31, 65, 1 << 20, 2 ** 31 - 1):
        with pytest.raises(g.NMSError) as e:
            g.route_experts(on_gpu(1 << 14, 128), k)
        assert e.value.status == "NMS_INVALID_ARG"
