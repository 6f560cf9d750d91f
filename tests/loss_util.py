"""Inputs and error bounds shared by the GPU tests of the losses.

The bounds count roundings of 2^-24 (U), with x = (m - z) / t of a logit, p its
probability and X1, X2 the sums of p x and p x^2 of a row:

* an exponential: the difference, the product and its factor are rounded
  (3 U x, and U x for the factor's own constant), the instruction is good to an
  ulp (2 U): (4 x + 2) U of its value;
* a sum: N additions in a row, N = vocab / 256 + 64 at most (a thread of 256
  adds its own, then lanes, waves and slices): s is off by (4 X1 + 2 + N) U;
* a log probability: that of log s, 3 U of (m - z) / t, and its own rounding;
* an entropy log s - ln 2 w / s: w's terms have 2 U more each;
* a gradient p (...) / t: its exponential, 1 / s and six products and sums;
  then once to the logits' type, half a step of it.  An exponential below
  2^-126 of the largest is 0 (the instruction has no subnormal results), which
  takes at most 2^-126 of (...) / t off, as s is 1 at least.
"""
import numpy as np

from gpu_util import device

import torch

from oracle import losses as plain

U = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]
# the smallest normal numbers of a type are its subnormals' scale
SMALL = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}


def lib():
    import greedy_iou_nms_amd as g
    return g


def dev(a, dtype=None):
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(device())


def host(t):
    return t.detach().double().cpu().numpy()


def logits_of(rng, T, V, dtype, spread=3.0, stride=None, shift=0):
    """Random logits of a type, as a matrix of this row stride whose first
    element is `shift` elements past an aligned address."""
    z = torch.from_numpy((spread * rng.normal(size=(T, V))).astype(np.float32)).to(dtype)
    if stride is None and shift == 0:
        return z.to(device())
    stride = V if stride is None else stride
    space = torch.full((T * stride + shift + 16,), float("nan"), dtype=dtype)
    view = space[shift:shift + T * stride].view(T, stride)[:, :V]
    view.copy_(z)
    return space.to(device())[shift:shift + T * stride].view(T, stride)[:, :V]


class Bounds:
    """What the results of rows may be off by, from their logits in 64 bits."""

    def __init__(self, z, tokens, temperature=None, weights=None):
        z = np.asarray(z, np.float64)
        T, V = z.shape
        self.n = V / 256 + 64
        self.counts, self.lp, self.h, self.dlp, self.dh = plain.rows(z, tokens, temperature,
                                                                     weights)
        self.t = np.array([plain.temperature_of(temperature, r) for r in range(T)])
        with np.errstate(all="ignore"):
            top = np.max(np.where(np.isnan(z), -np.inf, z), axis=1, keepdims=True)
            x = np.where(z > -np.inf, (top - z) / self.t[:, None], np.inf)
            y = np.stack([plain.log_softmax(z[r], self.t[r]) for r in range(T)])
            p = np.exp(y)
            self.x = np.where(p > 0, x, 0.0)
            self.s0 = np.full(T, np.log(V))  # log s at most
            self.y = np.where(p > 0, y, 0.0)
        self.p = np.where(np.isfinite(p), p, 0.0)
        x1, x2 = (self.p * self.x).sum(1), (self.p * self.x ** 2).sum(1)
        self.s = U * (4 * x1 + 2 + self.n)
        at = np.clip(np.asarray(tokens), 0, V - 1)
        xa = np.where(np.isfinite(x), x, 0.0)[np.arange(T), at]
        fin = lambda v: np.where(np.isfinite(v), np.abs(v), 0.0)
        self.logprob = self.s + U * (3 * xa + fin(self.lp)) + 2.0 ** -126
        self.entropy = self.s + x1 * self.s + U * (x1 * (self.n + 4) + 4 * x2 + fin(self.h))

    def grad(self, dtype, want, g, h=None, dg=0.0):
        """Of the gradient `want` from g and h in a row's results, g off by dg."""
        g = np.abs(np.where(self.counts, g, 0.0))[:, None]
        h = np.zeros_like(g) if h is None else np.abs(np.where(self.counts, h, 0.0))[:, None]
        rel = U * (4 * self.x + 8) + self.s[:, None]
        per = self.p / self.t[:, None]
        size = per * (g + h * (np.abs(self.y) + self.h[:, None]))
        err = rel * size + per * h * self.entropy[:, None]
        y = np.where(np.isfinite(self.x), self.x, 0.0) + self.s0[:, None]
        err += 2.0 ** -126 * (g + h * (y + self.h[:, None])) / self.t[:, None]
        err += np.abs(self.dlp) * (np.broadcast_to(dg, self.lp.shape)[:, None] + 3 * U * g)
        half = torch.finfo(dtype).eps / 2
        return np.nan_to_num(err * (1 + half) + half * np.abs(want)) + SMALL[dtype]


def within(got, want, tol, what=""):
    """NaN and infinities alike, and everything else within its bound."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    wild = ~np.isfinite(want)
    assert np.array_equal(got[wild & ~np.isnan(want)], want[wild & ~np.isnan(want)]), what
    with np.errstate(invalid="ignore"):
        err = np.where(wild, 0.0, np.abs(got - want))
    tol = np.broadcast_to(tol, want.shape)
    bad = ~(err <= tol)
    assert not bad.any(), (what, err[bad][:4], tol[bad][:4], np.argwhere(bad)[:4])
