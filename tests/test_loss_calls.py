"""What the binding of the losses hands to the library, without a GPU: the
library's entry points are replaced by ones that note their arguments, and the
tensors only claim to be on a GPU."""
import ctypes

import pytest
import torch

import greedy_iou_nms_amd as g
from greedy_iou_nms_amd import losses as mod


class Claimed(torch.Tensor):
    is_cuda = True


def on_gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Claimed)


def plain_fields(struct):
    return {name: getattr(struct, name) for name, _ in struct._fields_}


class Library:
    """Notes the arguments of each call, the options as they are at the call."""
    OPTIONS = {"nms_policy_loss": (11, mod._PolicyOptions),
               "nms_preference_loss": (10, mod._PreferenceOptions),
               "nms_preference_loss_backward": (9, mod._PreferenceOptions),
               "nms_balance_loss": (9, mod._BalanceOptions)}

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace_size"):
                ctypes.cast(args[-1], ctypes.POINTER(ctypes.c_size_t)).contents.value = 4096
                return 0
            options = None
            if name in self.OPTIONS:
                at, kind = self.OPTIONS[name]
                options = plain_fields(ctypes.cast(args[at], ctypes.POINTER(kind)).contents)
            self.calls.append((name, args, options))
            return 0
        return call

    def last(self):
        return self.calls[-1]


@pytest.fixture
def library(monkeypatch):
    fake = Library()
    monkeypatch.setattr(mod, "_lib", fake)
    monkeypatch.setattr(mod, "_current_device", lambda: None)  # a CPU device's index
    monkeypatch.setattr(mod, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(mod, "_capturing", lambda: False)
    caches = (mod._loss_workspace_size, mod._balance_workspace_size)
    for c in caches:
        c.cache_clear()
    yield fake
    for c in caches:
        c.cache_clear()  # the sizes here are made up


def rows(T=3, V=11):
    return on_gpu(T, V), on_gpu(T, dtype=torch.int32), on_gpu(T), on_gpu(T)


def close(a, b):
    return a == pytest.approx(b, rel=1e-6)


def test_policy_options(library):
    z, a, old, adv = rows()
    g.policy_loss(z, a, old, adv)
    assert library.last()[2] == pytest.approx(dict(clip_low=0.2, clip_high=0.2, kl=0, entropy=0))
    g.policy_loss(z, a, old, adv, clip=0.1, clip_high=0.3, kl=0.5, entropy=-0.25,
                  ref_logprobs=on_gpu(3))
    assert library.last()[2] == pytest.approx(dict(clip_low=0.1, clip_high=0.3, kl=0.5,
                                                   entropy=-0.25))
    # numbers, not their holders
    clip = torch.tensor(0.5)
    for value in (0.5, 0.25):
        clip.fill_(value)
        g.policy_loss_with_grad(z, a, old, adv, clip=clip)
        assert library.last()[2]["clip_low"] == library.last()[2]["clip_high"] == value


def test_policy_outputs(library):
    z, a, old, adv = rows()
    for entropy, n in ((None, 2), (0.0, 3), (0.1, 3)):
        assert len(g.policy_loss(z, a, old, adv, entropy=entropy)) == n
        args = library.last()[1]
        assert (args[15] is None) == (entropy is None)          # entropies
        assert args[16] is None                                  # gradient
        got = g.policy_loss_with_grad(z, a, old, adv, entropy=entropy)
        assert len(got) == n + 1
        args = library.last()[1]
        assert args[13:17] == (got[0].data_ptr(), got[2].data_ptr(),
                               None if entropy is None else got[3].data_ptr(), got[1].data_ptr())
        assert args[17] == 11 and args[12] is None


def test_rows_and_strides(library):
    wide = on_gpu(3, 40)
    z, (_, a, old, adv) = wide[:, 5:16], rows()
    heat, w, ref, up = on_gpu(3), on_gpu(3), on_gpu(3), on_gpu(1)
    out = on_gpu(3, 50)[:, :11]
    g.policy_loss_with_grad(z, a, old, adv, w, ref, heat, kl=0.1, grad_loss=up, out=out)
    args = library.last()[1]
    assert args[:6] == (z.data_ptr(), 0, 3, 11, 40, a.data_ptr())
    assert args[6:11] == tuple(t.data_ptr() for t in (old, adv, w, ref, heat))
    assert args[12] == up.data_ptr() and args[16:18] == (out.data_ptr(), 50)
    g.token_logprobs_backward(z.half(), a, old, heat, adv)
    args = library.last()[1]
    assert args[1:5] == (1, 3, 11, 11)
    assert args[6:9] == (heat.data_ptr(), old.data_ptr(), adv.data_ptr())


def test_preference_calls(library):
    z, a, _, _ = rows(6)
    at = on_gpu(5, dtype=torch.int64)
    got = g.preference_loss(z, a, at, beta=0.5, kind="squared", margin=0.25, average=True)
    name, args, options = library.last()
    assert name == "nms_preference_loss" and args[6:8] == (at.data_ptr(), 2)
    assert options == pytest.approx(dict(kind=2, average=1, beta=0.5, smoothing=0, margin=0.25))
    assert [t.shape for t in got] == [(), (4,), (2,)] and args[15] is None
    g.preference_loss_with_grad(z, a, at, smoothing=0.125)
    assert library.last()[2]["smoothing"] == 0.125 and library.last()[1][16] == 11


def test_balance_calls(library):
    z, ids = on_gpu(6, 8), on_gpu(6, 2, dtype=torch.int32)
    loss, counts = g.balance_loss(z, ids, "sigmoid", balance=0.5, z=0.25)
    name, args, options = library.last()
    assert options == dict(score=1, top_k=2, balance=0.5, z=0.25) and counts.shape == (8,)
    assert args[5:9] == (ids.data_ptr(), None, None, 1) and args[12] == counts.data_ptr()
    at = on_gpu(4, dtype=torch.int64)
    loss, dz, counts = g.balance_loss_with_grad(z, ids, offsets=at, live=on_gpu(6).bool())
    assert counts.shape == (3, 8) and library.last()[1][7:9] == (at.data_ptr(), 3)
    loss, dz, same = g.balance_loss_with_grad(z, counts=counts, offsets=at)
    args = library.last()[1]
    assert same is counts and args[5] is None and args[12] == counts.data_ptr()
    # ids without a place, or without rows, are ids all the same
    g.balance_loss(z, ids[:, :0])
    assert library.last()[1][5] is not None
    g.balance_loss(z[:0], ids[:0])
    assert library.last()[1][5] is not None


def test_workspaces(library, monkeypatch):
    """Kept between calls, apart from those of other operators; a captured call
    has one of its own."""
    z, a, old, adv = rows()
    g.token_logprobs(z, a)
    first = library.last()[1][9]
    g.policy_loss(z, a, old, adv)
    assert library.last()[1][18] == first and library.last()[1][19] == 4096
    cpu = torch.device("cpu")
    for use in ("nms", "pick"):
        buf = g._default_workspace(cpu, 0, use).get(1 << 16, cpu)
        assert not buf.data_ptr() <= first < buf.data_ptr() + buf.numel()
    monkeypatch.setattr(mod, "_capturing", lambda: True)
    kept = []
    get = g.Workspace.get
    monkeypatch.setattr(g.Workspace, "get",
                        lambda self, n, d: kept.append(get(self, n, d)) or kept[-1])
    g.token_logprobs(z, a)
    g.token_logprobs(z, a)
    assert kept[0].data_ptr() != kept[1].data_ptr() and first not in (
        kept[0].data_ptr(), kept[1].data_ptr())


def test_unused_outputs_and_an_upstream_of_the_wrong_kind(library):
    z, a, old, adv = rows()
    assert isinstance(g.token_logprobs(z, a), torch.Tensor)
    assert len(g.token_logprobs(z, a, entropy=True)) == 2
    with pytest.raises(TypeError):
        g.policy_loss_with_grad(z, a, old, adv, grad_loss=1.0)
    assert not library.calls[2:]


def test_tangents_are_refused(library):
    """Forward-mode differentiation has no part in the calls: an input with a
    tangent is refused, not stripped of it, whether or not gradients are recorded."""
    z, a, old, adv = rows(6)
    two, pair, up = on_gpu(2), on_gpu(1), on_gpu(1)
    at, ids = on_gpu(3, dtype=torch.int64), on_gpu(6, 2, dtype=torch.int32)
    calls = [(g.token_logprobs, [z, a, adv]),
             (g.token_logprobs_backward, [z, a, old, adv, old]),
             (g.policy_loss, [z, a, old, adv, adv, old, adv]),
             (g.policy_loss_with_grad, [z, a, old, adv, adv, old, adv]),
             (lambda *v: g.policy_loss_with_grad(*v[:-1], grad_loss=v[-1]), [z, a, old, adv, up]),
             (g.preference_loss, [z, a, at, two, pair]),
             (g.preference_loss_with_grad, [z, a, at, two, pair]),
             (lambda *v: g.preference_loss_with_grad(*v[:-1], grad_loss=v[-1]), [z, a, at, up]),
             (g.balance_loss, [z, ids]), (g.balance_loss_with_grad, [z, ids]),
             (lambda *v: g.balance_loss_with_grad(*v[:-1], grad_loss=v[-1]), [z, ids, up])]
    forward = torch.autograd.forward_ad
    for call, args in calls:
        with forward.dual_level():
            call(*args)                     # nothing here has one
            for i, t in enumerate(args):
                if not t.is_floating_point():
                    continue
                with_tangent = list(args)
                with_tangent[i] = forward.make_dual(t, torch.ones_like(t))
                made = len(library.calls)
                with pytest.raises(RuntimeError, match="tangent"):
                    call(*with_tangent)
                with torch.no_grad(), pytest.raises(RuntimeError, match="tangent"):
                    call(*with_tangent)
                assert len(library.calls) == made
        call(*args)
    with forward.dual_level():
        out = forward.make_dual(on_gpu(6, 11), on_gpu(6, 11))
        with pytest.raises(RuntimeError, match="tangent"):
            g.policy_loss_with_grad(z, a, old, adv, out=out)
        leaf = on_gpu(6, 11).requires_grad_()
        with pytest.raises((RuntimeError, NotImplementedError)):
            g.token_logprobs(forward.make_dual(leaf, torch.ones_like(leaf)), a)
