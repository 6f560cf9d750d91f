"""Plain 64-bit implementations of the losses of language models (log
probabilities of given tokens, policy loss, preference loss, balance loss of
routing) with their gradients, row by row from the definitions in
``include/greedy_nms.h``.  Test infrastructure: numpy only, no code shared with
the library.
"""
from __future__ import annotations

import numpy as np


def log_softmax(z, t=1.0):
    """log softmax(z / t) of one row, -infinity throughout where no logit is
    above it; NaN where one is NaN or +infinity.  At t = infinity all logits
    above -infinity weigh alike."""
    z = np.asarray(z, np.float64)
    if np.isnan(z).any() or np.isposinf(z).any():
        return np.full_like(z, np.nan)
    there = z > -np.inf
    out = np.full_like(z, -np.inf)
    if there.any():
        y = np.zeros(there.sum()) if np.isinf(t) else (z[there] - z[there].max()) / t
        out[there] = y - np.log(np.exp(y).sum())
    return out


def temperature_of(temperature, row):
    t = 1.0 if temperature is None else float(temperature[row])
    return t if t > 0 else 1.0


def _row(z, token, t):
    """(log probability, entropy, their gradients in the row)."""
    y = log_softmax(z, t)
    p = np.exp(y)
    if not (p.sum() > 0):
        if np.isnan(y).any():
            return np.nan, np.nan, np.full_like(p, np.nan), np.full_like(p, np.nan)
        return -np.inf, 0.0, np.zeros_like(p), np.zeros_like(p)
    ylogy = np.where(p > 0, p * np.where(p > 0, y, 0.0), 0.0)
    h = -ylogy.sum()
    one = np.zeros_like(p)
    one[token] = 1.0
    return y[token], h, (one - p) / t, -(ylogy + p * h) / t


def rows(logits, tokens, temperature=None, weights=None):
    """Per row: whether it counts, log probability, entropy and their gradients
    (rows, vocab)."""
    logits = np.asarray(logits, np.float64)
    T, V = logits.shape
    counts = (np.asarray(tokens) >= 0) & (np.asarray(tokens) < V)
    if weights is not None:
        counts &= ~(np.asarray(weights) == 0)
    lp, h = np.zeros(T), np.zeros(T)
    dlp, dh = np.zeros((T, V)), np.zeros((T, V))
    for r in np.flatnonzero(counts):
        lp[r], h[r], dlp[r], dh[r] = _row(logits[r], tokens[r], temperature_of(temperature, r))
    return counts, lp, h, dlp, dh


def combine(counts, dlp, dh, g, h):
    """The gradient in the logits from those in log probability and entropy; a
    row whose two are 0 has none."""
    g = np.where(counts, g, 0.0)
    h = np.where(counts, 0.0 if h is None else h, 0.0)
    out = np.zeros_like(dlp)
    for r in np.flatnonzero((g != 0) | (h != 0)):
        out[r] = g[r] * dlp[r] + (h[r] * dh[r] if h[r] != 0 else 0.0)
    return out


def policy(logits, tokens, old, advantages, weights=None, ref=None, temperature=None, clip=0.2,
           clip_high=None, kl=0.0, entropy=0.0, up=1.0):
    """(loss, logprobs, entropies, gradient in the logits, in log probability,
    in entropy)."""
    counts, lp, h, dlp, dh = rows(logits, tokens, temperature, weights)
    T = len(lp)
    high = clip if clip_high is None else clip_high
    loss, g, e = 0.0, np.zeros(T), np.zeros(T)
    for r in np.flatnonzero(counts):
        w = 1.0 / T if weights is None else float(weights[r])
        A = float(advantages[r])
        ratio = np.exp(lp[r] - float(old[r]))
        each = slope = 0.0
        if A != 0:
            free, held = ratio * A, min(max(ratio, 1 - clip), 1 + high) * A
            if np.isnan(free):
                each = slope = np.nan
            else:
                each = -min(free, held)
                slope = -free if free <= held else 0.0
        if kl:
            q = float(ref[r]) - lp[r]
            each += kl * (np.expm1(q) - q)
            slope -= kl * np.expm1(q)
        each -= entropy * h[r] if entropy else 0.0
        loss += w * each
        g[r], e[r] = up * w * slope, -up * w * entropy
    return loss, lp, h, combine(counts, dlp, dh, g, e), g, e


def starts(offsets, n):
    """Where sequences start and end: the largest offset so far, within n rows."""
    return np.clip(np.maximum.accumulate(np.maximum(np.asarray(offsets), 0)), 0, n)


def preference(logits, tokens, offsets, ref=None, weights=None, beta=0.1, kind="sigmoid",
               smoothing=0.0, margin=0.0, average=False, up=1.0):
    """(loss, logprobs, margins, gradient in the logits, in log probability)."""
    counts, lp, _, dlp, dh = rows(logits, tokens)
    at = starts(offsets, len(lp))
    P = (len(at) - 1) // 2
    sums, sizes = np.zeros(2 * P), np.ones(2 * P)
    for q in range(2 * P):
        own = slice(at[q], at[q + 1])
        if average:
            sizes[q] = max(1, counts[own].sum())
        sums[q] = lp[own][counts[own]].sum() / sizes[q]
    loss, margins, g = 0.0, np.zeros(P), np.zeros(len(lp))
    for i in range(P):
        r = np.zeros(2) if ref is None else np.asarray(ref, np.float64)[[i, P + i]]
        h = beta * ((sums[i] - r[0]) - (sums[P + i] - r[1])) - margin
        margins[i] = h
        w = 1.0 / P if weights is None else float(weights[i])
        if kind == "sigmoid":
            each = (1 - smoothing) * np.logaddexp(0, -h)
            each += smoothing * np.logaddexp(0, h) if smoothing else 0.0
            slope = smoothing / (1 + np.exp(-h)) - (1 - smoothing) / (1 + np.exp(h))
        elif kind == "hinge":
            each, slope = max(0.0, 1 - h), -1.0 if h < 1 else 0.0
            if np.isnan(h):
                each = slope = h
        else:
            each, slope = ((h - 0.5) / beta) ** 2, 2 * (h - 0.5) / beta ** 2
        if w == 0:
            continue
        loss += w * each
        for q, sign in ((i, 1.0), (P + i, -1.0)):
            g[at[q]:at[q + 1]] = sign * up * w * slope * beta / sizes[q]
    return loss, sums, margins, combine(counts, dlp, dh, g, None), np.where(counts, g, 0.0)


def balance(logits, ids=None, score="softmax", balance=1.0, z=0.0, offsets=None, live=None,
            counts=None, up=1.0):
    """(loss, counts, gradient in the logits)."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    at = np.array([0, T]) if offsets is None else starts(offsets, T)
    S = len(at) - 1
    alive = np.ones(T, bool) if live is None else np.asarray(live).astype(bool)
    given = counts is not None
    counts = np.maximum(np.asarray(counts).reshape(S, E), 0) if given else np.zeros((S, E), np.int64)
    loss, dz = 0.0, np.zeros((T, E))
    used = np.zeros(T, bool)
    for q in range(S):
        mine = [t for t in range(at[q], at[q + 1]) if alive[t]]
        used[mine] = True
        if not given:
            for t in mine:
                for e in ids[t]:
                    if 0 <= e < E:
                        counts[q, e] += 1
        if not mine or counts[q].sum() == 0:
            f = np.zeros(E)
        else:
            f = E * counts[q] / counts[q].sum()
        for t in mine:
            row = logits[t]
            if np.isnan(row).any():
                loss = np.nan
                dz[t] = np.nan
                continue
            there = row > -np.inf
            if not there.any():
                continue
            if score == "softmax":
                s = np.exp(log_softmax(row))
                rest = np.ones(E)
            else:
                # shares of sigmoids by their logarithms, -log(1 + exp(-z))
                logs = np.where(there, -np.logaddexp(0, -np.where(there, row, 0.0)), -np.inf)
                s = np.exp(logs - logs[there].max())
                s = s / s.sum()
                rest = 1.0 / (1.0 + np.exp(np.where(there, row, 0.0)))
            a = balance / S * f / len(mine)
            loss += (a * s).sum()
            dz[t] += s * rest * (a - (a * s).sum())
    n = used.sum()
    if z:
        for t in np.flatnonzero(used):
            row = logits[t]
            there = row > -np.inf
            if not there.any() or np.isnan(row).any():
                continue
            top = row.max()
            lse = top + np.log(np.exp(row[there] - top).sum())
            loss += z / n * lse ** 2
            dz[t] += 2 * z / n * lse * np.exp(log_softmax(row))
    return loss, counts.astype(np.int32), up * dz
