"""Selection operators of language models: routing to experts, rules on
logits and picking the next token (the ``nms_route_*``, ``nms_adjust_logits``
and ``nms_pick_tokens`` entry points of ``include/greedy_nms.h``, which states
what each computes).

Like the rest of the binding: tensor checks, output allocation, pointers and
the current HIP stream of the tensors' device.  The calls do not wait for the
GPU and may be captured into a graph (a captured call takes its workspace
from the graph's own memory).
"""
from __future__ import annotations

import ctypes
import functools
import operator
from typing import Optional, Tuple

import torch

from . import Workspace, _check, _default_workspace, _lib, _raw_stream

_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_capturing = torch.cuda.is_current_stream_capturing
# tells autograd that a tensor's values change, which the library does unseen
_overwritten = torch.autograd.graph.increment_version
_data_ptr, _size, _stride = torch.Tensor.data_ptr, torch.Tensor.size, torch.Tensor.stride

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}  # nms_dtype
_SCORES = {"softmax": 0, "sigmoid": 1}  # NMS_ROUTE_SOFTMAX, NMS_ROUTE_SIGMOID
_MAX_EXPERTS_PER_TOKEN = 64  # NMS_ROUTE_MAX_TOP_K


class _RouteOptions(ctypes.Structure):  # nms_route_options
    _fields_ = [("score", ctypes.c_int), ("top_k", ctypes.c_int), ("renormalise", ctypes.c_int),
                ("scale", ctypes.c_float), ("groups", ctypes.c_int),
                ("kept_groups", ctypes.c_int), ("group_top", ctypes.c_int)]


class _LogitRules(ctypes.Structure):  # nms_logit_rules
    _fields_ = [("history", ctypes.c_void_p), ("history_stride", ctypes.c_int64),
                ("history_capacity", ctypes.c_int64), ("history_len", ctypes.c_void_p),
                ("prompt_len", ctypes.c_void_p), ("repetition", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("bias_ids", ctypes.c_void_p), ("bias_values", ctypes.c_void_p),
                ("bias_stride", ctypes.c_int64), ("bias_count", ctypes.c_int64),
                ("allowed", ctypes.c_void_p), ("allowed_stride", ctypes.c_int64),
                ("allowed_count", ctypes.c_int64), ("allowed_rows", ctypes.c_void_p)]


def _address(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _matrix(t, name: str) -> Tuple[int, int, int, int]:
    """(nms_dtype, rows, columns, row stride) of a matrix of a floating type on
    a GPU device.  The checks are those of _rows, which says what is wrong."""
    try:
        rows, columns = t.shape
        stride, inner = t.stride()
        code = _DTYPES[t.dtype]
    except (AttributeError, KeyError, TypeError, ValueError):
        code = None
    if code is None or not t.is_cuda or inner != 1 or (rows > 1 and stride < columns):
        stride = _rows(t, name)
        rows, columns = t.shape
        code = _DTYPES[t.dtype]
    return code, rows, columns, stride


def _like(logits, rows: int, columns: int, stride: int) -> torch.Tensor:
    """A contiguous matrix of the logits' shape and type (1 us less of the
    caller's time where they are contiguous themselves)."""
    if stride == columns:
        return torch.empty_like(logits)
    return torch.empty((rows, columns), dtype=logits.dtype, device=logits.device)


def _rows(t, name: str, device=None, shape=None, dtype=None) -> int:
    """The row stride of a matrix whose rows hold neighbouring elements and
    do not overlap; other layouts are refused."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dim() != 2:
        raise ValueError("%s must be a matrix" % name)
    if dtype is None:
        if t.dtype not in _DTYPES:
            raise TypeError("%s must be float32, float16 or bfloat16 (got %s)" % (name, t.dtype))
    elif t.dtype is not dtype:
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if device is None:
        if not t.is_cuda:
            raise ValueError("%s must be on a GPU device" % name)
    elif t.device != device:
        raise ValueError("%s must be on %s (got %s)" % (name, device, t.device))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    rows, columns = t.shape
    if rows > 0 and columns > 1 and t.stride(1) != 1:
        raise ValueError("%s must have neighbouring elements in a row" % name)
    stride = t.stride(0)
    if rows > 1 and stride < columns:
        raise ValueError("the rows of %s overlap" % name)
    return stride if rows > 1 else columns


def _vector(t, name: str, n: int, dtype, device) -> Optional[int]:
    """The address of a contiguous vector of n elements, or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if (t.dtype is dtype and t.device == device and t.shape == (n,) and
            (n < 2 or t.stride() == (1,))):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s must be on %s (got %s)" % (name, device, t.device))
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError("%s must have shape (%d,)" % (name, n))
    raise ValueError("%s must be contiguous" % name)


def _whole(v, name: str, bits: int = 32) -> int:
    """A plain integer; ctypes would cut what its C type does not hold."""
    v = operator.index(v)
    if not -1 << (bits - 1) <= v < 1 << (bits - 1):
        raise ValueError("%s is out of range (got %d)" % (name, v))
    return v


# ------------------------------------------------------------------- routing

def _route_options(score, top_k, renormalise, scale, groups, kept_groups, group_top):
    """The options' address.  They are remembered by plain numbers: a tensor
    would be remembered by its identity, whatever it holds by the next call,
    and 4.0 be taken for a 4 of an earlier one."""
    if not (type(top_k) is type(groups) is type(group_top) is int and type(scale) is float and
            (kept_groups is None or type(kept_groups) is int)):
        top_k, groups, group_top = map(operator.index, (top_k, groups, group_top))
        kept_groups = None if kept_groups is None else operator.index(kept_groups)
        scale = float(scale)
    return _plain_options(score, top_k, bool(renormalise), scale, groups, kept_groups, group_top)


@functools.lru_cache(maxsize=256)
def _plain_options(score, top_k, renormalise, scale, groups, kept_groups, group_top):
    if score not in _SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid' (got %r)" % (score,))
    kept_groups = groups if kept_groups is None else kept_groups
    return ctypes.byref(_RouteOptions(
        _SCORES[score], _whole(top_k, "top_k"), int(renormalise), scale, _whole(groups, "groups"),
        _whole(kept_groups, "kept_groups"), _whole(group_top, "group_top")))


def route_experts(logits: torch.Tensor, top_k: int, score: str = "softmax",
                  bias: Optional[torch.Tensor] = None, groups: int = 1,
                  kept_groups: Optional[int] = None, group_top: int = 2,
                  renormalise: bool = True, scale: float = 1.0,
                  live: Optional[torch.Tensor] = None, counts: bool = False):
    """The experts of every token and their weights: ``(ids, weights)``, int32
    and float32 tensors of shape (tokens, top_k); with ``counts=True`` also an
    int32 tensor of how many tokens chose each expert.

    ``logits`` is a (tokens, experts) tensor; ``bias`` (float32, one per
    expert) counts for the choice only; of ``groups`` groups of neighbouring
    experts ``kept_groups`` (default: all) may be chosen from; ``live`` (bool
    or uint8, one per token) marks padded rows with 0.  A place that no expert
    is left for holds id -1 and weight 0.

    Where ``logits`` require a gradient, the weights carry it
    (``route_experts_backward``).  While a step is captured with its backward
    pass, no eager graph of the same leaves may be alive, as with torch's own
    operators."""
    code, tokens, experts, stride = _matrix(logits, "logits")
    device = logits.device
    if logits.requires_grad and torch.is_grad_enabled():
        return _Routed.apply(logits, top_k, score, bias, groups, kept_groups, group_top,
                             bool(renormalise), float(scale), live, counts)
    if type(top_k) is not int:
        top_k = operator.index(top_k)  # of the options and of the outputs
    if device.index != _current_device():
        with torch.cuda.device(device):
            return route_experts(logits, top_k, score, bias, groups, kept_groups, group_top,
                                 renormalise, scale, live, counts)
    options = _route_options(score, top_k, renormalise, scale, groups, kept_groups, group_top)
    b = None if bias is None else _vector(bias, "bias", experts, torch.float32, device)
    alive = None if live is None else _vector(
        live, "live", tokens, torch.bool if getattr(live, "dtype", None) is torch.bool
        else torch.uint8, device)
    # a top_k that the library will refuse gets no outputs
    shape = (tokens, top_k if 0 < top_k <= _MAX_EXPERTS_PER_TOKEN else 0)
    ids = torch.empty(shape, dtype=torch.int32, device=device)
    weights = torch.empty(shape, dtype=torch.float32, device=device)
    count = torch.empty(experts, dtype=torch.int32, device=device) if counts else None
    status = _lib.nms_route_experts(logits.data_ptr(), code, tokens, experts, stride, b, alive,
                                    options, ids.data_ptr(), weights.data_ptr(),
                                    _address(count), _raw_stream(device))
    if status:
        _check(status)
    return (ids, weights, count) if counts else (ids, weights)


class _Routed(torch.autograd.Function):
    """``route_experts`` (called without gradients here) and its gradient."""

    @staticmethod
    def forward(ctx, logits, top_k, score, bias, groups, kept_groups, group_top, renormalise,
                scale, live, counts):
        out = route_experts(logits, top_k, score, bias, groups, kept_groups, group_top,
                            renormalise, scale, live, counts)
        ctx.save_for_backward(logits, out[0])
        ctx.options = score, renormalise, scale
        ctx.mark_non_differentiable(out[0], *out[2:])
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_ids, grad_weights, *grad_counts):
        logits, ids = ctx.saved_tensors
        grad = route_experts_backward(logits, ids, grad_weights.contiguous(), *ctx.options)
        return (grad,) + (None,) * 10


def route_experts_backward(logits: torch.Tensor, ids: torch.Tensor, grad_weights: torch.Tensor,
                           score: str = "softmax", renormalise: bool = True, scale: float = 1.0,
                           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of ``route_experts``' weights in its logits, from the
    forward call's ``ids`` and the gradient of its weights; a tensor like
    ``logits`` (or ``out``, which may be ``logits`` itself, must not overlap it
    otherwise and is refused where it requires a gradient).  The choice of the
    experts, and so the bias, has no gradient, and this one has no further."""
    code, tokens, experts, stride = _matrix(logits, "logits")
    device = logits.device
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be a matrix of shape (tokens, top_k)")
    top_k = ids.shape[1]
    if not (ids.dtype is torch.int32 and ids.device == device and ids.is_contiguous() and
            ids.shape[0] == tokens and isinstance(grad_weights, torch.Tensor) and
            grad_weights.dtype is torch.float32 and grad_weights.device == device and
            grad_weights.shape == ids.shape and grad_weights.is_contiguous()):
        shape = torch.Size((tokens, top_k))
        _rows(ids, "ids", device, shape, torch.int32)
        _rows(grad_weights, "grad_weights", device, shape, torch.float32)
        raise ValueError("ids and grad_weights must be contiguous")
    if device.index != _current_device():
        with torch.cuda.device(device):
            return route_experts_backward(logits, ids, grad_weights, score, renormalise, scale,
                                          out)
    options = _route_options(score, top_k, renormalise, scale, 1, 1, 1)
    if out is None:
        out = _like(logits, tokens, experts, stride)
        out_stride = experts
    else:
        out_stride = _rows(out, "out", device, logits.shape, logits.dtype)
        if out.requires_grad and torch.is_grad_enabled():
            raise RuntimeError("route_experts_backward with an out that requires a gradient")
        _overwritten(out)
    status = _lib.nms_route_experts_backward(
        logits.data_ptr(), code, tokens, experts, stride, ids.data_ptr(), grad_weights.data_ptr(),
        options, out.data_ptr(), out_stride, _raw_stream(device))
    if status:
        _check(status)
    return out


# -------------------------------------------------------------------- logits

class LogitRules:
    """The rules of a batch of rows of logits (``nms_logit_rules``): penalties
    for tokens of the history, biases and masks of allowed tokens.

    A serving loop makes one and keeps it while the contents of its tensors
    change from step to step; it holds on to the tensors and their memory.  A
    matrix that has another shape by the next call, or a tensor with other
    memory (``resize_``, ``set_``, ``.data``), is checked anew and read where it
    is then; a captured graph goes on reading what it was captured with.  All
    tensors are on one device, with one row (or entry) per row of logits:

    ``history`` (rows, capacity) int32, the prompt and then what was
    generated; ``history_len`` and ``prompt_len`` (rows,) int32;
    ``repetition``, ``presence``, ``frequency`` (rows,) float32; ``bias_ids``
    int32 and ``bias_values`` float32, (rows, entries), ids outside the
    vocabulary unused; ``allowed`` (masks, words) int64, bit v mod 64 of word
    v // 64 for token v; ``allowed_rows`` (rows,) int32, the mask of each row
    (negative: every token is allowed).  None of them gets a gradient."""

    def __init__(self, vocab: int, history=None, history_len=None, prompt_len=None,
                 repetition=None, presence=None, frequency=None, bias_ids=None, bias_values=None,
                 allowed=None, allowed_rows=None):
        self.vocab = int(vocab)
        self._given = (history, history_len, prompt_len, repetition, presence, frequency,
                       bias_ids, bias_values, allowed, allowed_rows)
        self._lay_out()

    def _lay_out(self) -> None:
        """Checks the tensors and takes down where they are."""
        (history, history_len, prompt_len, repetition, presence, frequency, bias_ids, bias_values,
         allowed, allowed_rows) = self._given
        per_row = (history, history_len, prompt_len, repetition, presence, frequency, bias_ids,
                   bias_values, allowed_rows)
        if allowed is not None and allowed_rows is None:
            per_row += (allowed,)
        given = [t for t in self._given if t is not None]
        if not all(isinstance(t, torch.Tensor) and t.dim() > 0 for t in given):
            raise TypeError("the rules must be torch tensors with a dimension")
        # before anything is read of them
        matrices = [t for t in (history, bias_ids, bias_values, allowed) if t is not None]
        addresses, shapes = list(map(_data_ptr, given)), list(map(_size, matrices))
        strides = list(map(_stride, matrices))
        device = given[0].device if given else None
        if given and not given[0].is_cuda:
            raise ValueError("the rules must be on a GPU device")
        rows = {t.shape[0] for t in per_row if t is not None}
        if len(rows) > 1:
            raise ValueError("the rules have different numbers of rows: %s" % sorted(rows))
        n = rows.pop() if rows else None
        if (history is None) != (history_len is None):
            raise ValueError("history and history_len go together")
        if prompt_len is not None and history is None:
            raise ValueError("prompt_len goes with a history")
        if (bias_ids is None) != (bias_values is None):
            raise ValueError("bias_ids and bias_values go together")
        if allowed_rows is not None and allowed is None:
            raise ValueError("allowed_rows goes with masks of allowed tokens")
        c = _LogitRules()
        if history is not None:
            c.history_stride = _rows(history, "history", device, None, torch.int32)
            c.history, c.history_capacity = history.data_ptr(), history.shape[1]
            c.history_len = _vector(history_len, "history_len", n, torch.int32, device)
            c.prompt_len = _vector(prompt_len, "prompt_len", n, torch.int32, device)
            # an empty history has no address
            if history.shape[1] == 0:
                c.history = c.history_len = c.prompt_len = None
        c.repetition = _vector(repetition, "repetition", n, torch.float32, device)
        c.presence = _vector(presence, "presence", n, torch.float32, device)
        c.frequency = _vector(frequency, "frequency", n, torch.float32, device)
        if bias_ids is not None:
            c.bias_stride = _rows(bias_ids, "bias_ids", device, None, torch.int32)
            if _rows(bias_values, "bias_values", device, bias_ids.shape,
                     torch.float32) != c.bias_stride:
                raise ValueError("bias_ids and bias_values must have the same strides")
            c.bias_ids, c.bias_values = bias_ids.data_ptr(), bias_values.data_ptr()
            c.bias_count = bias_ids.shape[1]
        if allowed is not None:
            c.allowed_stride = _rows(allowed, "allowed", device, None, torch.int64)
            if allowed.shape[1] < (self.vocab + 63) // 64:
                raise ValueError("allowed must have %d words per mask" % ((self.vocab + 63) // 64))
            # an empty table has no address; it is never read, but the
            # numbers of its masks count
            c.allowed, c.allowed_count = allowed.data_ptr() or 8, allowed.shape[0]
            c.allowed_rows = _vector(allowed_rows, "allowed_rows", n, torch.int32, device)
        self.device, self.rows = device, n
        self._struct = c
        self._ref = ctypes.byref(c)
        # aliases hold the memory that the addresses are of
        self._memory = [t.detach() for t in given]
        self._tensors, self._addresses = given, addresses
        self._matrices, self._shapes, self._strides = matrices, shapes, strides

    def _for(self, rows: int, vocab: int, device) -> object:
        """The struct's address, for logits of this shape."""
        # (a vector whose memory is the same is read for as many rows as it had)
        if (list(map(_data_ptr, self._tensors)) != self._addresses or
                list(map(_size, self._matrices)) != self._shapes or
                list(map(_stride, self._matrices)) != self._strides):
            self._lay_out()
        if self.vocab != vocab:
            raise ValueError("the rules are for %d tokens, the logits have %d" % (self.vocab, vocab))
        if self.rows is not None and self.rows != rows:
            raise ValueError("the rules are for %d rows, the logits have %d" % (self.rows, rows))
        if self.device is not None and self.device != device:
            raise ValueError("the rules must be on %s (got %s)" % (device, self.device))
        return self._ref


class _Ungraded(torch.autograd.Function):
    """The outputs of a call that has no gradient here, though its logits
    require one: a backward pass that reaches them raises, where it would go on
    without their part."""

    @staticmethod
    def forward(ctx, logits, name, call):
        out = call(logits)
        ctx.name = name
        if isinstance(out, tuple):
            ctx.mark_non_differentiable(*(t for t in out if not t.is_floating_point()))
        return out

    @staticmethod
    def backward(ctx, *grads):
        raise NotImplementedError("%s has no gradient" % ctx.name)


def _rules(rules, rows: int, vocab: int, device) -> object:
    if not isinstance(rules, LogitRules):
        raise TypeError("rules must be LogitRules")
    return rules._for(rows, vocab, device)


def adjust_logits(logits: torch.Tensor, rules: LogitRules,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The logits under the rules, a tensor like ``logits`` (or ``out``, which
    may be ``logits`` itself and must not overlap it otherwise).  It has no
    gradient: a backward pass through it raises, and ``out`` is refused where
    it or the logits require one."""
    code, rows, vocab, stride = _matrix(logits, "logits")
    device = logits.device
    if ((logits.requires_grad or (out is not None and getattr(out, "requires_grad", False))) and
            torch.is_grad_enabled()):
        if out is not None:
            raise RuntimeError("adjust_logits with out has no gradient, but logits or out "
                               "require one")
        return _Ungraded.apply(logits, "adjust_logits", lambda z: adjust_logits(z, rules))
    ref = _rules(rules, rows, vocab, device)
    if device.index != _current_device():
        with torch.cuda.device(device):
            return adjust_logits(logits, rules, out)
    if out is None:
        out = _like(logits, rows, vocab, stride)
        out_stride = vocab
    else:
        out_stride = _rows(out, "out", device, logits.shape, logits.dtype)
        _overwritten(out)
    status = _lib.nms_adjust_logits(logits.data_ptr(), code, rows, vocab, stride, ref,
                                    out.data_ptr(), out_stride, _raw_stream(device))
    if status:
        _check(status)
    return out


def pick_workspace_size(rows: int, vocab: int, max_top_k: int) -> int:
    """The bytes of workspace that ``pick_tokens`` takes."""
    return _pick_workspace_size(_whole(rows, "rows", 64), _whole(vocab, "vocab", 64),
                                _whole(max_top_k, "max_top_k"))


@functools.lru_cache(maxsize=256)
def _pick_workspace_size(rows: int, vocab: int, max_top_k: int) -> int:
    # a function of the sizes alone, so it can be remembered
    out = ctypes.c_size_t(0)
    _check(_lib.nms_pick_workspace_size(rows, vocab, max_top_k, ctypes.byref(out)))
    return int(out.value)


def pick_tokens(logits: torch.Tensor, uniform: torch.Tensor, max_top_k: int = 64,
                temperature: Optional[torch.Tensor] = None, top_k: Optional[torch.Tensor] = None,
                top_p: Optional[torch.Tensor] = None, min_p: Optional[torch.Tensor] = None,
                rules: Optional[LogitRules] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The next token of every row of ``logits`` under the rules: ``(ids,
    logprobs)``, int32 and float32 tensors of shape (rows,).

    ``uniform`` (rows,) float32 holds one number in [0, 1) per row;
    ``temperature`` (0: the first token), ``top_p`` and ``min_p`` are float32
    and ``top_k`` int32, one per row.  The draw is always from the first
    ``max_top_k`` tokens (64 unless given, at most 1024) or a row's first
    ``top_k`` of them; a ``top_k`` of 0 or below takes the first token and does
    not lift the limit.  The logprob is that of the token under the softmax over all
    allowed tokens.  A row without an allowed token gets -1 and -infinity.
    The logprobs have no gradient: a backward pass through them raises."""
    code, rows, vocab, stride = _matrix(logits, "logits")
    device = logits.device
    if logits.requires_grad and torch.is_grad_enabled():
        return _Ungraded.apply(logits, "pick_tokens", lambda z: pick_tokens(
            z, uniform, max_top_k, temperature, top_k, top_p, min_p, rules))
    if uniform is None:
        raise TypeError("uniform must be a torch tensor")
    f32 = torch.float32
    u = _vector(uniform, "uniform", rows, f32, device)
    t = None if temperature is None else _vector(temperature, "temperature", rows, f32, device)
    k = None if top_k is None else _vector(top_k, "top_k", rows, torch.int32, device)
    p = None if top_p is None else _vector(top_p, "top_p", rows, f32, device)
    m = None if min_p is None else _vector(min_p, "min_p", rows, f32, device)
    ref = None if rules is None else _rules(rules, rows, vocab, device)
    if device.index != _current_device():
        with torch.cuda.device(device):
            return pick_tokens(logits, uniform, max_top_k, temperature, top_k, top_p, min_p,
                               rules)
    max_top_k = _whole(max_top_k, "max_top_k")
    nbytes = _pick_workspace_size(rows, vocab, max_top_k)
    # kept per thread and stream; a captured call takes one of its own from
    # the graph's memory, so that no two graphs share it
    stream = _raw_stream(device)
    kept = Workspace(device) if _capturing() else _default_workspace(device, stream, "pick")
    buf = kept.get(nbytes, device)
    ids = torch.empty(rows, dtype=torch.int32, device=device)
    logprobs = torch.empty_like(uniform)
    status = _lib.nms_pick_tokens(logits.data_ptr(), code, rows, vocab, stride, ref, u, t, k, p, m,
                                  max_top_k, ids.data_ptr(), logprobs.data_ptr(),
                                  buf.data_ptr(), nbytes, stream)
    if status:
        _check(status)
    return ids, logprobs
