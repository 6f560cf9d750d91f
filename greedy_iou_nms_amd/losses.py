"""Losses of language models: log probabilities of given tokens, the clipped
policy loss and the preference loss made of them, and the balance loss of
routing, with their gradients (the ``nms_token_logprobs``, ``nms_policy_loss``,
``nms_preference_loss`` and ``nms_balance_loss`` entry points of
``include/greedy_nms.h``, which states what each computes).

Each loss comes in two forms.  ``policy_loss`` and the like carry their
gradient through autograd.  ``policy_loss_with_grad`` and the like return the
gradient in the logits with the loss, from one call that need not read the
logits a second time (``torch.autograd.backward(logits, grad)`` takes it from
there).  Gradients have none of their own, and inputs with a tangent (of
forward-mode differentiation) are refused.  The calls do not wait for the GPU
and may be captured into a graph; while a step is captured with its backward
pass, no eager graph of the same leaves may be alive, as with torch's own
operators.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad as _forward

from . import Workspace, _check, _default_workspace, _lib, _raw_stream
from .selection import (_SCORES, _address, _capturing, _current_device, _like, _matrix,
                        _overwritten, _rows, _vector, _whole)

_KINDS = {"sigmoid": 0, "hinge": 1, "squared": 2}  # NMS_PREFERENCE_*


class _PolicyOptions(ctypes.Structure):  # nms_policy_options
    _fields_ = [("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float),
                ("kl", ctypes.c_float), ("entropy", ctypes.c_float)]


class _PreferenceOptions(ctypes.Structure):  # nms_preference_options
    _fields_ = [("kind", ctypes.c_int), ("average", ctypes.c_int), ("beta", ctypes.c_float),
                ("smoothing", ctypes.c_float), ("margin", ctypes.c_float)]


class _BalanceOptions(ctypes.Structure):  # nms_balance_options
    _fields_ = [("score", ctypes.c_int), ("top_k", ctypes.c_int), ("balance", ctypes.c_float),
                ("z", ctypes.c_float)]


# (options are remembered by plain numbers only)

@functools.lru_cache(maxsize=256)
def _policy_options(clip, clip_high, kl, entropy):
    return ctypes.byref(_PolicyOptions(clip, clip_high, kl, entropy))


@functools.lru_cache(maxsize=256)
def _preference_options(kind, average, beta, smoothing, margin):
    if kind not in _KINDS:
        raise ValueError("kind must be 'sigmoid', 'hinge' or 'squared' (got %r)" % (kind,))
    return ctypes.byref(_PreferenceOptions(_KINDS[kind], average, beta, smoothing, margin))


@functools.lru_cache(maxsize=256)
def _balance_options(score, top_k, balance, z):
    if score not in _SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid' (got %r)" % (score,))
    return ctypes.byref(_BalanceOptions(_SCORES[score], top_k, balance, z))


@functools.lru_cache(maxsize=256)
def _loss_workspace_size(rows: int, vocab: int, pairs: int) -> int:
    # a function of the sizes alone, so it can be remembered
    out = ctypes.c_size_t(0)
    _check(_lib.nms_loss_workspace_size(rows, vocab, pairs, ctypes.byref(out)))
    return int(out.value)


@functools.lru_cache(maxsize=256)
def _balance_workspace_size(tokens: int, experts: int, sequences: int, top_k: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.nms_balance_workspace_size(tokens, experts, sequences, top_k, ctypes.byref(out)))
    return int(out.value)


def _space(nbytes: int, device, stream: int) -> torch.Tensor:
    """A workspace, kept per thread and stream; a captured call takes one of its
    own from the graph's memory, so that no two graphs share it."""
    kept = Workspace(device) if _capturing() else _default_workspace(device, stream, "loss")
    return kept.get(nbytes, device)


def _constant(name: str, **tensors) -> None:
    """Refuses tensors that require a gradient, which the call does not have."""
    if torch.is_grad_enabled():
        for key, t in tensors.items():
            if t is not None and getattr(t, "requires_grad", False):
                raise RuntimeError("%s has no gradient in %s, which requires one"
                                   % (name, key))


def _no_tangents(name: str, *tensors) -> None:
    """Refuses tensors with a tangent, which the outputs would lack.  (They have
    one within a level of forward-mode differentiation only.)"""
    for t in tensors:
        if isinstance(t, torch.Tensor) and _forward.unpack_dual(t).tangent is not None:
            raise RuntimeError("%s has no forward-mode gradient: an input has a tangent" % name)


def _float(t, name: str, n: int, device) -> Optional[int]:
    return None if t is None else _vector(t, name, n, torch.float32, device)


def _upstream(grad_loss, device) -> Optional[int]:
    """The address of the loss's gradient, a float32 tensor of one element."""
    if grad_loss is None:
        return None
    if not isinstance(grad_loss, torch.Tensor):
        raise TypeError("grad_loss must be a torch tensor")
    if grad_loss.dtype is not torch.float32:
        raise TypeError("grad_loss must be torch.float32 (got %s)" % grad_loss.dtype)
    if grad_loss.device != device:
        raise ValueError("grad_loss must be on %s (got %s)" % (device, grad_loss.device))
    if grad_loss.numel() != 1:
        raise ValueError("grad_loss must have one element")
    return grad_loss.data_ptr()


def _gradient_of(logits, rows: int, columns: int, stride: int, out, name: str):
    """Where a gradient in the logits goes, and its row stride."""
    if out is None:
        return _like(logits, rows, columns, stride), columns
    out_stride = _rows(out, "out", logits.device, logits.shape, logits.dtype)
    if out.requires_grad and torch.is_grad_enabled():
        raise RuntimeError("%s with an out that requires a gradient" % name)
    _overwritten(out)
    return out, out_stride


def _graph(logits) -> bool:
    return logits.requires_grad and torch.is_grad_enabled()


def _scalar(device) -> torch.Tensor:
    return torch.empty((), dtype=torch.float32, device=device)


# --------------------------------------------------- log probabilities of tokens

def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor,
                   temperature: Optional[torch.Tensor] = None, entropy: bool = False):
    """The log probabilities of given tokens, a float32 tensor of shape (rows,);
    with ``entropy=True`` also the entropies of the rows.

    ``tokens`` (rows,) int32 holds a token per row of ``logits``; a row whose
    token is outside the vocabulary (-1, say) does not count: it has log
    probability and entropy 0 and is not read.  ``temperature`` (rows,) float32
    divides the logits, as in ``pick_tokens``.  Where ``logits`` require a
    gradient, both outputs carry it (``token_logprobs_backward``)."""
    code, rows, vocab, stride = _matrix(logits, "logits")
    device = logits.device
    _constant("token_logprobs", temperature=temperature)
    if _forward._current_level >= 0:
        _no_tangents("token_logprobs", logits, temperature)
    if _graph(logits):
        got = _TokenLogprobs.apply(logits, tokens, temperature, bool(entropy))
        return got if entropy else got[0]
    if tokens is None:
        raise TypeError("tokens must be a torch tensor")
    a = _vector(tokens, "tokens", rows, torch.int32, device)
    t = _float(temperature, "temperature", rows, device)
    if device.index != _current_device():
        with torch.cuda.device(device):
            return token_logprobs(logits, tokens, temperature, entropy)
    nbytes = _loss_workspace_size(rows, vocab, 0)
    stream = _raw_stream(device)
    logprobs = torch.empty(rows, dtype=torch.float32, device=device)
    entropies = torch.empty_like(logprobs) if entropy else None
    space = _space(nbytes, device, stream)
    status = _lib.nms_token_logprobs(logits.data_ptr(), code, rows, vocab, stride, a, t,
                                     logprobs.data_ptr(), _address(entropies),
                                     space.data_ptr(), nbytes, stream)
    if status:
        _check(status)
    return (logprobs, entropies) if entropy else logprobs


class _TokenLogprobs(torch.autograd.Function):
    """``token_logprobs`` (called without gradients here) and its gradient."""

    @staticmethod
    def forward(ctx, logits, tokens, temperature, entropy):
        got = token_logprobs(logits, tokens, temperature, entropy)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(logits, tokens, temperature)
        return got if entropy else (got,)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_logprobs, grad_entropies=None):
        logits, tokens, temperature = ctx.saved_tensors
        if grad_logprobs is None and grad_entropies is None:
            return (None,) * 4
        if grad_logprobs is None:
            grad_logprobs = torch.zeros_like(grad_entropies)
        grad = token_logprobs_backward(
            logits, tokens, grad_logprobs.contiguous(), temperature,
            None if grad_entropies is None else grad_entropies.contiguous())
        return grad, None, None, None


def token_logprobs_backward(logits: torch.Tensor, tokens: torch.Tensor,
                            grad_logprobs: torch.Tensor,
                            temperature: Optional[torch.Tensor] = None,
                            grad_entropies: Optional[torch.Tensor] = None,
                            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of ``token_logprobs`` in its logits, from those of the log
    probabilities and of the entropies; a tensor like ``logits`` (or ``out``,
    which may be ``logits`` itself, must not overlap it otherwise and is
    refused where it requires a gradient).  A row whose two gradients are 0 has
    gradient 0, whatever it holds."""
    code, rows, vocab, stride = _matrix(logits, "logits")
    device = logits.device
    if _forward._current_level >= 0:
        _no_tangents("token_logprobs_backward", logits, grad_logprobs, temperature,
                     grad_entropies, out)
    if tokens is None or grad_logprobs is None:
        raise TypeError("tokens and grad_logprobs must be torch tensors")
    a = _vector(tokens, "tokens", rows, torch.int32, device)
    g = _vector(grad_logprobs, "grad_logprobs", rows, torch.float32, device)
    t = _float(temperature, "temperature", rows, device)
    h = _float(grad_entropies, "grad_entropies", rows, device)
    if device.index != _current_device():
        with torch.cuda.device(device):
            return token_logprobs_backward(logits, tokens, grad_logprobs, temperature,
                                           grad_entropies, out)
    nbytes = _loss_workspace_size(rows, vocab, 0)
    out, out_stride = _gradient_of(logits, rows, vocab, stride, out, "token_logprobs_backward")
    stream = _raw_stream(device)
    space = _space(nbytes, device, stream)
    status = _lib.nms_token_logprobs_backward(
        logits.data_ptr(), code, rows, vocab, stride, a, t, g, h, out.data_ptr(), out_stride,
        space.data_ptr(), nbytes, stream)
    if status:
        _check(status)
    return out


# ------------------------------------------------------------------ policy loss

def _run_policy(logits, tokens, old_logprobs, advantages, weights, ref_logprobs, temperature,
                clip, clip_high, kl, entropy, grad_loss, results: bool, gradient: bool, out,
                name: str):
    """(loss, grad_logits, logprobs, entropies), None what is not asked for."""
    code, rows, vocab, stride = _matrix(logits, "logits")
    device = logits.device
    if _forward._current_level >= 0:
        _no_tangents(name, logits, old_logprobs, advantages, weights, ref_logprobs, temperature,
                     grad_loss, out)
    if tokens is None or old_logprobs is None or advantages is None:
        raise TypeError("tokens, old_logprobs and advantages must be torch tensors")
    a = _vector(tokens, "tokens", rows, torch.int32, device)
    old = _float(old_logprobs, "old_logprobs", rows, device)
    adv = _float(advantages, "advantages", rows, device)
    w = _float(weights, "weights", rows, device)
    ref = _float(ref_logprobs, "ref_logprobs", rows, device)
    t = _float(temperature, "temperature", rows, device)
    up = _upstream(grad_loss, device)
    options = _policy_options(float(clip), float(clip if clip_high is None else clip_high),
                              float(kl), 0.0 if entropy is None else float(entropy))
    if device.index != _current_device():
        with torch.cuda.device(device):
            return _run_policy(logits, tokens, old_logprobs, advantages, weights, ref_logprobs,
                               temperature, clip, clip_high, kl, entropy, grad_loss, results,
                               gradient, out, name)
    nbytes = _loss_workspace_size(rows, vocab, 0)
    grad, grad_stride = (_gradient_of(logits, rows, vocab, stride, out, name) if gradient
                         else (None, 0))
    loss = _scalar(device) if results else None
    logprobs = torch.empty_like(old_logprobs) if results else None
    entropies = torch.empty_like(old_logprobs) if results and entropy is not None else None
    stream = _raw_stream(device)
    space = _space(nbytes, device, stream)
    status = _lib.nms_policy_loss(
        logits.data_ptr(), code, rows, vocab, stride, a, old, adv, w, ref, t, options, up,
        _address(loss), _address(logprobs), _address(entropies), _address(grad), grad_stride,
        space.data_ptr(), nbytes, stream)
    if status:
        _check(status)
    return loss, grad, logprobs, entropies


def policy_loss(logits: torch.Tensor, tokens: torch.Tensor, old_logprobs: torch.Tensor,
                advantages: torch.Tensor, weights: Optional[torch.Tensor] = None,
                ref_logprobs: Optional[torch.Tensor] = None,
                temperature: Optional[torch.Tensor] = None, clip: float = 0.2,
                clip_high: Optional[float] = None, kl: float = 0.0,
                entropy: Optional[float] = None):
    """The clipped policy loss of tokens that an earlier policy picked: ``(loss,
    logprobs)``, a float32 scalar and the tokens' log probabilities; with
    ``entropy`` (the weight of the entropy bonus, 0.0 for none) also the
    entropies of the rows.

    ``old_logprobs``, ``advantages``, ``weights`` (1 / rows unless given),
    ``ref_logprobs`` (needed for a ``kl`` above 0) and ``temperature`` are
    float32, ``tokens`` int32, one per row of ``logits``.  The ratio is held in
    1 - ``clip`` .. 1 + ``clip_high`` (``clip`` unless given).  A row of weight
    0, or whose token is outside the vocabulary, does not count and is not
    read; the weights make whatever mean is wanted.

    The loss carries its gradient in the logits, and the other outputs have
    none (``token_logprobs`` has)."""
    _constant("policy_loss", old_logprobs=old_logprobs, advantages=advantages, weights=weights,
              ref_logprobs=ref_logprobs, temperature=temperature)
    given = (tokens, old_logprobs, advantages, weights, ref_logprobs, temperature)
    options = (clip, clip_high, kl, entropy)
    if isinstance(logits, torch.Tensor) and _graph(logits):
        got = _PolicyLoss.apply(logits, *given, *options)
    else:
        loss, _, logprobs, entropies = _run_policy(logits, *given, *options, None, True, False,
                                                   None, "policy_loss")
        got = (loss, logprobs, entropies)
    return got if entropy is not None else got[:2]


def policy_loss_with_grad(logits: torch.Tensor, tokens: torch.Tensor, old_logprobs: torch.Tensor,
                          advantages: torch.Tensor, weights: Optional[torch.Tensor] = None,
                          ref_logprobs: Optional[torch.Tensor] = None,
                          temperature: Optional[torch.Tensor] = None, clip: float = 0.2,
                          clip_high: Optional[float] = None, kl: float = 0.0,
                          entropy: Optional[float] = None,
                          grad_loss: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None):
    """``policy_loss`` and the gradient of ``grad_loss`` (a float32 tensor of one
    element; None: 1) times the loss in the logits, in one call: ``(loss,
    grad_logits, logprobs)``, with ``entropy`` also the entropies.  The gradient
    is a tensor like ``logits``, or ``out`` (as for
    ``token_logprobs_backward``); none of them carries a graph."""
    got = _run_policy(logits, tokens, old_logprobs, advantages, weights, ref_logprobs,
                      temperature, clip, clip_high, kl, entropy, grad_loss, True, True, out,
                      "policy_loss_with_grad")
    return got if entropy is not None else got[:3]


class _PolicyLoss(torch.autograd.Function):

    @staticmethod
    def forward(ctx, logits, tokens, old, advantages, weights, ref, temperature, clip, clip_high,
                kl, entropy):
        given = (tokens, old, advantages, weights, ref, temperature)
        ctx.options = (float(clip), None if clip_high is None else float(clip_high), float(kl),
                       None if entropy is None else float(entropy))
        loss, _, logprobs, entropies = _run_policy(logits, *given, *ctx.options, None, True, False,
                                                   None, "policy_loss")
        ctx.save_for_backward(logits, *given)
        ctx.mark_non_differentiable(*(t for t in (logprobs, entropies) if t is not None))
        return loss, logprobs, entropies

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss, *unused):
        got = _run_policy(*ctx.saved_tensors, *ctx.options, grad_loss, False, True, None,
                          "policy_loss")
        return (got[1],) + (None,) * 10


# -------------------------------------------------------------- preference loss

def _run_preference(logits, tokens, offsets, ref_logprobs, weights, options, grad_loss, margins,
                    gradient: bool, out, name: str):
    """(loss, grad_logits, logprobs, margins); the gradient alone from known
    margins."""
    code, rows, vocab, stride = _matrix(logits, "logits")
    device = logits.device
    if _forward._current_level >= 0:
        _no_tangents(name, logits, ref_logprobs, weights, grad_loss, out)
    if tokens is None:
        raise TypeError("tokens must be a torch tensor")
    if not isinstance(offsets, torch.Tensor):
        raise TypeError("offsets must be a torch tensor")
    if offsets.dim() != 1 or offsets.shape[0] < 3 or offsets.shape[0] % 2 == 0:
        raise ValueError("offsets must have shape (2 * pairs + 1,), for one pair at least")
    n = offsets.shape[0] - 1
    a = _vector(tokens, "tokens", rows, torch.int32, device)
    at = _vector(offsets, "offsets", n + 1, torch.int64, device)
    ref = _float(ref_logprobs, "ref_logprobs", n, device)
    w = _float(weights, "weights", n // 2, device)
    up = _upstream(grad_loss, device)
    if device.index != _current_device():
        with torch.cuda.device(device):
            return _run_preference(logits, tokens, offsets, ref_logprobs, weights, options,
                                   grad_loss, margins, gradient, out, name)
    ref_options = _preference_options(*options)
    nbytes = _loss_workspace_size(rows, vocab, n // 2)
    grad, grad_stride = (_gradient_of(logits, rows, vocab, stride, out, name) if gradient
                         else (None, 0))
    stream = _raw_stream(device)
    loss = logprobs = None
    if margins is None:
        loss = _scalar(device)
        logprobs = torch.empty(n, dtype=torch.float32, device=device)
        margins = torch.empty(n // 2, dtype=torch.float32, device=device)
        space = _space(nbytes, device, stream)
        status = _lib.nms_preference_loss(
            logits.data_ptr(), code, rows, vocab, stride, a, at, n // 2, ref, w, ref_options, up,
            loss.data_ptr(), logprobs.data_ptr(), margins.data_ptr(), _address(grad), grad_stride,
            space.data_ptr(), nbytes, stream)
    else:
        space = _space(nbytes, device, stream)
        status = _lib.nms_preference_loss_backward(
            logits.data_ptr(), code, rows, vocab, stride, a, at, n // 2, w, ref_options,
            margins.data_ptr(), up, grad.data_ptr(), grad_stride,
            space.data_ptr(), nbytes, stream)
    if status:
        _check(status)
    return loss, grad, logprobs, margins


def _plain_preference(kind, average, beta, smoothing, margin):
    return kind, bool(average), float(beta), float(smoothing), float(margin)


def preference_loss(logits: torch.Tensor, tokens: torch.Tensor, offsets: torch.Tensor,
                    ref_logprobs: Optional[torch.Tensor] = None,
                    weights: Optional[torch.Tensor] = None, beta: float = 0.1,
                    kind: str = "sigmoid", smoothing: float = 0.0, margin: float = 0.0,
                    average: bool = False) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The loss of paired log ratios: ``(loss, logprobs, margins)``, a float32
    scalar, the sequences' log probabilities (2 * pairs,) and the pairs' margins.

    The rows of ``logits`` are those of 2 * pairs sequences one after another,
    first the preferred one of each pair and then the other one of each;
    ``offsets`` (2 * pairs + 1,) int64 says where they start.  ``tokens``
    (rows,) int32: a row whose token is outside the vocabulary (of a prompt,
    say) does not count and is not read.  ``ref_logprobs`` (2 * pairs,) float32
    are the reference's, sums or with ``average`` means like the log
    probabilities themselves; ``weights`` (pairs,) float32 is 1 / pairs unless
    given.  ``kind`` is "sigmoid" (with ``smoothing`` of the labels), "hinge" or
    "squared"; ``margin`` is what the preferred one has to be better by.

    The loss carries its gradient in the logits, and the other outputs have
    none (``token_logprobs`` has)."""
    _constant("preference_loss", ref_logprobs=ref_logprobs, weights=weights)
    options = _plain_preference(kind, average, beta, smoothing, margin)
    if isinstance(logits, torch.Tensor) and _graph(logits):
        return _PreferenceLoss.apply(logits, tokens, offsets, ref_logprobs, weights, options)
    loss, _, logprobs, margins = _run_preference(logits, tokens, offsets, ref_logprobs, weights,
                                                 options, None, None, False, None,
                                                 "preference_loss")
    return loss, logprobs, margins


def preference_loss_with_grad(logits: torch.Tensor, tokens: torch.Tensor, offsets: torch.Tensor,
                              ref_logprobs: Optional[torch.Tensor] = None,
                              weights: Optional[torch.Tensor] = None, beta: float = 0.1,
                              kind: str = "sigmoid", smoothing: float = 0.0, margin: float = 0.0,
                              average: bool = False, grad_loss: Optional[torch.Tensor] = None,
                              out: Optional[torch.Tensor] = None):
    """``preference_loss`` and the gradient of ``grad_loss`` times the loss in the
    logits (see ``policy_loss_with_grad``): ``(loss, grad_logits, logprobs,
    margins)``."""
    options = _plain_preference(kind, average, beta, smoothing, margin)
    return _run_preference(logits, tokens, offsets, ref_logprobs, weights, options, grad_loss,
                           None, True, out, "preference_loss_with_grad")


class _PreferenceLoss(torch.autograd.Function):

    @staticmethod
    def forward(ctx, logits, tokens, offsets, ref, weights, options):
        loss, _, logprobs, margins = _run_preference(logits, tokens, offsets, ref, weights,
                                                     options, None, None, False, None,
                                                     "preference_loss")
        ctx.options = options
        ctx.save_for_backward(logits, tokens, offsets, ref, weights, margins)
        ctx.mark_non_differentiable(logprobs, margins)
        return loss, logprobs, margins

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss, *unused):
        logits, tokens, offsets, ref, weights, margins = ctx.saved_tensors
        got = _run_preference(logits, tokens, offsets, ref, weights, ctx.options, grad_loss,
                              margins, True, None, "preference_loss")
        return (got[1],) + (None,) * 5


# ----------------------------------------------------------------- balance loss

def _run_balance(logits, ids, counts, score, balance, z, offsets, live, grad_loss, results: bool,
                 gradient: bool, out, name: str):
    """(loss, grad_logits, counts)."""
    code, tokens, experts, stride = _matrix(logits, "logits")
    device = logits.device
    if _forward._current_level >= 0:
        _no_tangents(name, logits, grad_loss, out)
    sequences = 1
    if offsets is not None:
        if not isinstance(offsets, torch.Tensor):
            raise TypeError("offsets must be a torch tensor")
        if offsets.dim() != 1 or offsets.shape[0] < 2:
            raise ValueError("offsets must have shape (sequences + 1,), for one at least")
        sequences = offsets.shape[0] - 1
    at = None if offsets is None else _vector(offsets, "offsets", sequences + 1, torch.int64,
                                              device)
    shape = torch.Size((experts,) if offsets is None else (sequences, experts))
    top_k = chosen = None
    if (ids is None) == (counts is None):
        raise ValueError("either ids or counts must be given")
    if ids is not None:
        if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
            raise ValueError("ids must be a matrix of shape (tokens, top_k)")
        top_k = ids.shape[1]
        _rows(ids, "ids", device, torch.Size((tokens, top_k)), torch.int32)
        if not ids.is_contiguous():
            raise ValueError("ids must be contiguous")
        chosen = ids.data_ptr() or 8  # no tokens have no address
    else:
        if not isinstance(counts, torch.Tensor):
            raise TypeError("counts must be a torch tensor")
        if (counts.dtype is not torch.int32 or counts.device != device or
                counts.shape != shape or not counts.is_contiguous()):
            raise ValueError("counts must be a contiguous int32 tensor of shape %s on %s"
                             % (tuple(shape), device))
        top_k = 0
    alive = None if live is None else _vector(
        live, "live", tokens, torch.bool if getattr(live, "dtype", None) is torch.bool
        else torch.uint8, device)
    up = _upstream(grad_loss, device)
    options = _balance_options(score, top_k, float(balance), float(z))
    if device.index != _current_device():
        with torch.cuda.device(device):
            return _run_balance(logits, ids, counts, score, balance, z, offsets, live, grad_loss,
                                results, gradient, out, name)
    nbytes = _balance_workspace_size(tokens, experts, sequences, top_k)
    grad, grad_stride = (_gradient_of(logits, tokens, experts, stride, out, name) if gradient
                         else (None, 0))
    loss = _scalar(device) if results else None
    if counts is None and results:
        counts = torch.empty(shape, dtype=torch.int32, device=device)
    stream = _raw_stream(device)
    space = _space(nbytes, device, stream)
    status = _lib.nms_balance_loss(
        logits.data_ptr(), code, tokens, experts, stride, chosen, alive, at, sequences, options,
        up, _address(loss), _address(counts), _address(grad), grad_stride,
        space.data_ptr(), nbytes, stream)
    if status:
        _check(status)
    return loss, grad, counts


def balance_loss(logits: torch.Tensor, ids: Optional[torch.Tensor] = None,
                 score: str = "softmax", balance: float = 1.0, z: float = 0.0,
                 offsets: Optional[torch.Tensor] = None, live: Optional[torch.Tensor] = None,
                 counts: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The balance loss of routing: ``(loss, counts)``, a float32 scalar and how
    many tokens chose each expert, int32.

    ``logits`` (tokens, experts), ``score`` and ``live`` are those of
    ``route_experts`` and ``ids`` what it returned; instead of ``ids``, ``counts``
    may be given (summed over ranks or micro-batches, say).  ``balance`` is the
    weight of the balance term, ``z`` that of the mean square of the
    logits' log-sum-exp.  With ``offsets`` (sequences + 1,) int64 the experts
    are balanced within each sequence of tokens, and the counts have a row for
    each.

    The loss carries its gradient in the logits; the counts have none."""
    if isinstance(logits, torch.Tensor) and _graph(logits):
        return _BalanceLoss.apply(logits, ids, counts, score, float(balance), float(z), offsets,
                                  live)
    loss, _, counts = _run_balance(logits, ids, counts, score, balance, z, offsets, live, None,
                                   True, False, None, "balance_loss")
    return loss, counts


def balance_loss_with_grad(logits: torch.Tensor, ids: Optional[torch.Tensor] = None,
                           score: str = "softmax", balance: float = 1.0, z: float = 0.0,
                           offsets: Optional[torch.Tensor] = None,
                           live: Optional[torch.Tensor] = None,
                           counts: Optional[torch.Tensor] = None,
                           grad_loss: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None):
    """``balance_loss`` and the gradient of ``grad_loss`` times the loss in the
    logits (see ``policy_loss_with_grad``): ``(loss, grad_logits, counts)``."""
    return _run_balance(logits, ids, counts, score, balance, z, offsets, live, grad_loss, True,
                        True, out, "balance_loss_with_grad")


class _BalanceLoss(torch.autograd.Function):

    @staticmethod
    def forward(ctx, logits, ids, counts, score, balance, z, offsets, live):
        loss, _, got = _run_balance(logits, ids, counts, score, balance, z, offsets, live, None,
                                    True, False, None, "balance_loss")
        ctx.options = score, balance, z
        # the gradient goes by the counts
        ctx.save_for_backward(logits, got, offsets, live)
        ctx.mark_non_differentiable(got)
        return loss, got

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss, *unused):
        logits, counts, offsets, live = ctx.saved_tensors
        got = _run_balance(logits, None, counts, *ctx.options, offsets, live, grad_loss, False,
                           True, None, "balance_loss")
        return (got[1],) + (None,) * 7
