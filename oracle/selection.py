"""Plain 64-bit implementations of the selection operators (routing to
experts, its gradient, rules on logits, picking the next token), row by row
from the definitions in ``include/greedy_nms.h``.  Test infrastructure: numpy
only, no code shared with the library.
"""
from __future__ import annotations

import math

import numpy as np


def _first(values, n, allowed):
    """The indices of the n largest allowed values, ties to the lower index."""
    at = sorted((i for i in range(len(values)) if allowed[i]), key=lambda i: (-values[i], i))
    return at[:n]


def expert_scores(z, score):
    """softmax or sigmoid of one row; an expert with a NaN or -infinity logit
    has score 0 and no part in the sum."""
    z = np.asarray(z, np.float64)
    there = z > -np.inf
    s = np.zeros_like(z)
    if not there.any():
        return s, there
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "softmax":
            top = z[there].max()
            s[there] = np.where(z[there] == top, 1.0, np.exp(z[there] - top))
            s /= s.sum()
        else:
            s[there] = 1.0 / (1.0 + np.exp(-z[there]))
    return s, there


def route(logits, top_k, score="softmax", bias=None, groups=1, kept_groups=None, group_top=2,
          renormalise=True, scale=1.0, live=None):
    """(ids, weights, counts) as int32, float64, int32."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    kept_groups = groups if kept_groups is None else kept_groups
    ids = np.full((T, top_k), -1, np.int32)
    weights = np.zeros((T, top_k))
    for t in range(T):
        if live is not None and not live[t]:
            continue
        z = logits[t]
        s, there = expert_scores(z, score)
        with np.errstate(invalid="ignore"):
            c = s + (np.zeros(E) if bias is None else np.asarray(bias, np.float64))
        there = there & (c > -np.inf)
        if groups > 1:
            size = E // groups
            total = np.full(groups, -np.inf)
            some = np.zeros(groups, bool)
            for g in range(groups):
                part = range(g * size, (g + 1) * size)
                best = _first(c[part.start:part.stop], group_top, there[part.start:part.stop])
                some[g] = len(best) > 0
                total[g] = sum(c[part.start + i] for i in best)
            kept = set(_first(total, kept_groups, some))
            there = there & np.array([e // size in kept for e in range(E)])
        chosen = _first(z if bias is None else c, top_k, there)
        w = s[chosen]
        if renormalise and chosen:
            if score == "softmax":
                top = z[chosen].max()
                with np.errstate(invalid="ignore"):
                    w = np.where(z[chosen] == top, 1.0, np.exp(z[chosen] - top))
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = w * np.float64(np.float32(scale))
    counts = np.bincount(ids[ids >= 0], minlength=E).astype(np.int32)
    return ids, weights, counts


def route_backward(logits, ids, grad_weights, score="softmax", renormalise=True, scale=1.0):
    """The gradient (float64) and, per element, the sum of the absolute values
    of the terms it is made of (which its rounding errors are relative to)."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    grad, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        s, _ = expert_scores(logits[t], score)
        at = [i for i in range(ids.shape[1]) if 0 <= ids[t, i] < E]
        e = ids[t, at]
        g = np.asarray(grad_weights, np.float64)[t, at] * np.float64(np.float32(scale))
        q = s[e]
        total = q.sum()
        if len(at) == 0 or (renormalise and total == 0):
            continue
        if renormalise:
            mean = (g * q).sum() / total
            dq, dsize = (g - mean) / total, (abs(g) + (abs(g) * q).sum() / total) / total
        else:
            dq, dsize = g, abs(g)
        if score == "sigmoid":
            for i, j in enumerate(e):
                grad[t, j] += dq[i] * s[j] * (1.0 - s[j])
                size[t, j] += dsize[i] * s[j] * (1.0 - s[j])
            continue
        inner = 0.0 if renormalise else (dq * q).sum()
        grad[t] = -s * inner
        size[t] = s * (0.0 if renormalise else (dsize * q).sum())
        for i, j in enumerate(e):
            grad[t, j] += s[j] * dq[i]
            size[t, j] += s[j] * dsize[i]
    return grad, size


def adjust(logits, history=None, history_len=None, prompt_len=None, repetition=None,
           presence=None, frequency=None, bias_ids=None, bias_values=None, allowed=None,
           allowed_rows=None):
    """The adjusted logits in float32, one rounding a step, token by token."""
    z = np.array(logits, np.float32)
    B, V = z.shape
    f32 = np.float32
    with np.errstate(all="ignore"):
        for b in range(B):
            if history is not None:
                cap = history.shape[1]
                n = min(max(int(history_len[b]), 0), cap)
                p = 0 if prompt_len is None else min(max(int(prompt_len[b]), 0), n)
                tokens = [int(v) for v in history[b, :n]]
                r = f32(1.0) if repetition is None else f32(repetition[b])
                f = f32(0.0) if frequency is None else f32(frequency[b])
                q = f32(0.0) if presence is None else f32(presence[b])
                for v in set(tokens):
                    if 0 <= v < V:
                        z[b, v] = z[b, v] / r if z[b, v] > 0 else z[b, v] * r
                times = {}
                for v in tokens[p:]:
                    times[v] = times.get(v, 0) + 1
                for v, c in times.items():
                    if 0 <= v < V:
                        z[b, v] = f32(f32(z[b, v] - f32(f * f32(c))) - q)
            if bias_ids is not None:
                last = {}
                for v, x in zip(bias_ids[b], bias_values[b]):
                    last[int(v)] = f32(x)
                for v, x in last.items():
                    if 0 <= v < V:
                        z[b, v] = f32(z[b, v] + x)
            if allowed is not None:
                row = b if allowed_rows is None else int(allowed_rows[b])
                if row >= allowed.shape[0]:
                    z[b] = -np.inf
                elif row >= 0:
                    words = np.asarray(allowed)[row].astype(np.int64).view(np.uint64)
                    bits = np.unpackbits(words.view(np.uint8), bitorder="little")[:V]
                    z[b, bits == 0] = -np.inf
    return z


def pick(z, uniform, max_top_k, temperature=None, top_k=None, top_p=None, min_p=None):
    """(ids, logprobs) as int32 and float64 from adjusted float32 logits."""
    B, V = z.shape
    ids, logprobs = np.full(B, -1, np.int32), np.full(B, -np.inf)
    for b in range(B):
        x = z[b].astype(np.float64)
        there = np.flatnonzero(x > -np.inf)
        if there.size == 0:
            continue
        heat = 1.0 if temperature is None else float(np.float32(temperature[b]))
        t = heat if heat > 0 else 1.0
        k = max_top_k if top_k is None else min(max(int(top_k[b]), 1), max_top_k)
        order = there[np.argsort(-x[there], kind="stable")]
        top = x[order[0]]

        def weight(v):
            return 1.0 if v == top else math.exp(max((v - top) / t, -1e6))

        cand = order[:k]
        w = [weight(x[i]) for i in cand]
        p = 1.0 if top_p is None else float(np.float32(top_p[b]))
        m = 0.0 if min_p is None else float(np.float32(min_p[b]))
        n, running = 0, 0.0
        while n < len(w):
            running += w[n]
            n += 1
            if running >= p * math.fsum(w):
                break
        n = max(1, min(n, sum(v >= m for v in w)))
        bound, running, j = float(np.float32(uniform[b])) * math.fsum(w[:n]), 0.0, 0
        for j in range(n):
            running += w[j]
            if running > bound:
                break
        j = j if heat > 0 else 0
        ids[b] = cand[j]
        d = 0.0 if x[cand[j]] == top else (x[cand[j]] - top) / t
        logprobs[b] = d - math.log(math.fsum(weight(v) for v in x[there]))
    return ids, logprobs
