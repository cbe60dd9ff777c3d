"""Norms, products with an epilogue and balance losses of include/zc_moe.h in 64 bits,
written from their formulas with numpy, and what 32-bit sums may be off by."""
from __future__ import annotations

import math

import numpy as np

from moe_ref import BF16_HALF_STEP, F32_HALF_STEP, bf16  # noqa: F401

NONE, RMS, LAYER = range(3)
EPS32 = F32_HALF_STEP


def f32(x):
    return np.asarray(x, dtype=np.float32).astype(np.float64)


def stat(v, kind, eps):
    """mean and 1 / deviation of every row."""
    mu = v.mean(axis=1, keepdims=True) if kind == LAYER else np.zeros((v.shape[0], 1))
    return mu, 1 / np.sqrt(((v - mu) ** 2).mean(axis=1, keepdims=True) + eps)


def normed_error(v, mu, rs):
    """Bound on the 32-bit normed value: the difference to the mean loses 2 half steps of either and, with sums about 40
    additions deep, 40 of the mean deviation; the deviation's sum half of 42, its root 2."""
    hat = (v - mu) * rs
    return EPS32 * (2 * (np.abs(v) + np.abs(mu)) * rs + 64 * (1 + np.abs(hat)))


class Side:
    """One norm: kind, weight, bias (or None), eps."""

    def __init__(self, kind=NONE, w=None, b=None, eps=1e-6):
        self.kind, self.w, self.b, self.eps = kind, w, b, eps

    def apply(self, v, err=0.0):
        """(normed value, N(v), bound on its 32-bit error from an input off by `err`)."""
        if self.kind == NONE:
            return v, v, err + np.zeros_like(v)
        mu, rs = stat(v, self.kind, self.eps)
        hat = (v - mu) * rs
        e = normed_error(v, mu, rs)
        if np.ndim(err):
            e = e + rs * (err + err.mean(axis=1, keepdims=True)) + np.abs(hat) * rs * np.sqrt(
                (err ** 2).mean(axis=1, keepdims=True))
        w = 1.0 if self.w is None else self.w
        b = 0.0 if self.b is None else self.b
        out = hat * w + b
        return hat, out, np.abs(w) * e + 2 * EPS32 * (np.abs(hat * w) + np.abs(b))


def norm(x, z, after, before, gate, row_gate, scale):
    """(r, its error, y, its error) before any rounding to BF16."""
    if z is None:
        r, err = x, np.zeros_like(x)
    else:
        _, h, eh = after.apply(z)
        coef = scale * (1.0 if gate is None else gate) * (1.0 if row_gate is None else row_gate[:, None])
        r = x + coef * h
        err = np.abs(coef) * eh + 4 * EPS32 * np.abs(coef * h) + EPS32 * np.abs(r)
    _, y, ey = before.apply(r, err)
    return r, err, y, ey


def _slope(v, side, u):
    """Gradient at v from u at N(v), and the size of the terms that make it."""
    if side.kind == NONE:
        return u, np.abs(u), v
    mu, rs = stat(v, side.kind, side.eps)
    hat = (v - mu) * rs
    d = u * (1.0 if side.w is None else side.w)
    g = d - hat * (d * hat).mean(axis=1, keepdims=True)
    size = np.abs(d) + (1 + np.abs(hat)) * (np.abs(d) * (1 + np.abs(hat))).mean(axis=1, keepdims=True)
    if side.kind == LAYER:
        g = g - d.mean(axis=1, keepdims=True)
    # a mean far above the deviation costs as many times more
    amp = 1 + (np.abs(v) + np.abs(mu)).max(axis=1, keepdims=True) * rs / (1 + np.abs(hat).max(axis=1, keepdims=True))
    return rs * g, rs * size * amp, hat


# Terms of a gradient: normed values off by 64 half steps, means of products of two such, and about ten roundings.
TERMS = 256


def norm_backward(r, z, after, before, gate, row_gate, scale, dr, dy):
    """{name: (value, bound on the 32-bit error)}."""
    rows = r.shape[0]
    deep = rows + 64  # additions of a sum over the rows, at most
    out = {}
    g, size = np.zeros_like(r), np.zeros_like(r)
    if dr is not None:
        g, size = g + dr, size + np.abs(dr)
    zero = np.zeros(r.shape[1])
    for name in ("dw1", "db1", "dgate", "dw2", "db2"):
        out[name] = (zero, zero)
    if dy is not None:
        back, s, hat = _slope(r, before, dy)
        g, size = g + back, size + s
        if before.kind != NONE:
            mu, rs = stat(r, before.kind, before.eps)
            e = normed_error(r, mu, rs)
            out["dw2"] = ((dy * hat).sum(0), (np.abs(dy) * e).sum(0) + deep * EPS32 * np.abs(dy * hat).sum(0))
            out["db2"] = (dy.sum(0), deep * EPS32 * np.abs(dy).sum(0))
    err = TERMS * EPS32 * size
    out["dx"] = (g, err)
    out["drow_gate"] = (np.zeros(rows), np.zeros(rows))
    if z is None:
        return out
    one = np.ones(r.shape[1])
    gt = one if gate is None else gate
    rg = np.ones(rows) if row_gate is None else row_gate
    hat, h, eh = after.apply(z)
    coef = scale * gt * rg[:, None]
    dh, edh = coef * g, np.abs(coef) * (err + 4 * EPS32 * np.abs(g))
    t = scale * rg[:, None] * g * h
    et = np.abs(scale * rg[:, None]) * (err * np.abs(h) + np.abs(g) * eh) + 4 * EPS32 * np.abs(t)
    out["dgate"] = (t.sum(0), et.sum(0) + deep * EPS32 * np.abs(t).sum(0))
    t = scale * gt * g * h
    et = np.abs(scale * gt) * (err * np.abs(h) + np.abs(g) * eh) + 4 * EPS32 * np.abs(t)
    out["drow_gate"] = (t.sum(1), et.sum(1) + 64 * EPS32 * np.abs(t).sum(1))
    if after.kind != NONE:
        mu, rs = stat(z, after.kind, after.eps)
        e = normed_error(z, mu, rs)
        out["dw1"] = ((dh * hat).sum(0), (np.abs(dh) * e + edh * np.abs(hat)).sum(0) + deep * EPS32 * np.abs(dh * hat).sum(0))
        out["db1"] = (dh.sum(0), edh.sum(0) + deep * EPS32 * np.abs(dh).sum(0))
    back, s, _ = _slope(z, after, dh)
    _, se, _ = _slope(z, after, edh)  # the size is linear in the gradient's magnitude
    out["dz"] = (back, TERMS * EPS32 * s + se)
    return out


# -- activations ------------------------------------------------------------------------------------------------------

ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh", "sigmoid")
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1 / (1 + e), e / (1 + e))


def activation(v, act):
    """(value, slope) in 64 bits."""
    if act == 0:
        return v, np.ones_like(v)
    if act == 1:
        return np.maximum(v, 0.0), (v > 0).astype(np.float64)
    if act in (2, 5):
        s = _sigmoid(v)
        ds = s * _sigmoid(-v)
        return (v * s, s + v * ds) if act == 2 else (s, ds)
    if act == 3:
        c = 0.5 * _erfc(-v / math.sqrt(2))
        return v * c, c + v * np.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    k = 2 * math.sqrt(2 / math.pi)
    u = k * (v + 0.044715 * v ** 3)
    s = _sigmoid(u)
    return v * s, s + v * s * _sigmoid(-u) * k * (1 + 3 * 0.044715 * v * v)


def activation_error(v, act):
    """(of the value, of the slope): bounds on the 32-bit error for an exact input.  An exponential or an erfc of an
    argument a few half steps off is as many times |argument| off: up to v^2 (or its cube for the tanh form, where
    the value has not vanished); a slope is the sum of two terms whose sizes count."""
    value, _ = activation(v, act)
    grow = {0: 0, 1: 0, 2: np.abs(v), 3: v * v, 4: np.abs(v) + 0.08 * np.abs(v) ** 3, 5: np.abs(v)}[act]
    # right of 0 the exponential is beside a 1; not so in the sigmoid's slope, which is even: e^-|v| for large |v|, whose
    # argument is rounded with its constant, in its product and, as the square of a root, twice over: 3 |v| half steps
    k = (16 + 4 * np.where(v > 0, 1, np.minimum(grow, 400))) * EPS32
    ks = (16 + 4 * np.minimum(grow, 400)) * EPS32 if act == 5 else k
    size = {0: 1.0, 1: 1.0}.get(act)
    if size is None:
        s = np.abs(value) / np.maximum(np.abs(v), 1e-30) if act != 5 else value
        near = np.where(np.abs(v) < 1e-30, 1.0, s)
        second = np.abs(v) * near * (1 + np.abs(v)) * (1 + (0.3 * v * v if act == 4 else 0))
        size = near + np.where(v > 0, np.abs(v) * np.exp(-np.minimum(np.abs(v), 700)) * (1 + 0.3 * v * v) + 1.0, second)
        if act == 5:
            size = _sigmoid(-np.abs(v))
    return k * np.abs(value) + 2.0 ** -125, ks * size + 2.0 ** -125


# -- balance ----------------------------------------------------------------------------------------------------------

def spans(offsets, tokens):
    """The sequences that offsets name: clamped to 0..tokens and to ascending order."""
    b = np.maximum.accumulate(np.clip(np.asarray(offsets, dtype=np.int64), 0, tokens))
    return list(zip(b[:-1], b[1:]))


def scores(x, sigmoid):
    """(p, softmax, log-sum-exp with 0 for a row of -inf, 1 - sigmoid)."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        top = x.max(axis=1, keepdims=True)
        top = np.where(np.isneginf(top), 0.0, top)
        e = np.exp(x - top)
        total = e.sum(axis=1, keepdims=True)
        soft = np.where(total == 0, 0.0, e / np.where(total == 0, 1.0, total))
        lse = np.where(total[:, 0] == 0, 0.0, top[:, 0] + np.log(np.where(total[:, 0] == 0, 1.0, total[:, 0])))
        if not sigmoid:
            return soft, soft, lse, np.ones_like(soft)
        s = _sigmoid(x)
        return s / (s.sum(axis=1, keepdims=True) + 1e-20), soft, lse, _sigmoid(-x)


def balance(x, ids, mask, offsets, experts, top_k, sigmoid):
    """counts, used, loss, zloss."""
    t = x.shape[0]
    on = np.ones(t, dtype=bool) if mask is None else mask != 0
    p, _, lse, _ = scores(x, sigmoid)
    sp = spans(offsets, t)
    counts, used = np.zeros((len(sp), experts), dtype=np.int64), np.zeros(len(sp), dtype=np.int64)
    loss, z = np.zeros(len(sp)), np.zeros(len(sp))
    for s, (a, b) in enumerate(sp):
        rows = np.arange(a, b)[on[a:b]]
        used[s] = n = rows.size
        i = ids[rows].reshape(-1)
        counts[s] = np.bincount(i[(i >= 0) & (i < experts)], minlength=experts)
        if n:
            loss[s] = experts / (top_k * n * n) * (counts[s] * p[rows].sum(axis=0)).sum()
            z[s] = (lse[rows] ** 2).sum() / n
    return counts, used, loss, z


def balance_backward(x, mask, offsets, experts, top_k, sigmoid, counts, used, dloss, dz, add):
    """(gradient, size of its terms)."""
    t = x.shape[0]
    on = np.ones(t, dtype=bool) if mask is None else mask != 0
    p, soft, lse, rest = scores(x, sigmoid)
    g = np.zeros_like(x) if add is None else add.copy()
    size = np.abs(g)
    for s, (a, b) in enumerate(spans(offsets, t)):
        rows = np.arange(a, b)[on[a:b]]
        if not rows.size or used[s] <= 0:
            continue
        if dloss is not None:
            f = counts[s] * experts / (top_k * float(used[s]))
            q = p[rows]
            fp = (f * q).sum(axis=1, keepdims=True)
            g[rows] += dloss[s] / used[s] * q * (f - fp) * rest[rows]
            size[rows] += abs(dloss[s]) / used[s] * q * (f + fp) * rest[rows]
        if dz is not None:
            d = 2 * dz[s] / used[s] * lse[rows, None] * soft[rows]
            g[rows] += d
            size[rows] += np.abs(d)
    return g, size
