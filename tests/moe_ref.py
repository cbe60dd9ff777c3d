"""The mixture-of-experts operators of include/zc_moe.h in 64 bits, written from
their formulas with numpy: what the GPU tests compare with."""
from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3, E5M2 = 2, 3  # ZC_FP8_E4M3, ZC_FP8_E5M2
BF16_HALF_STEP = 2.0 ** -8  # torch.finfo(torch.bfloat16).eps / 2
F32_HALF_STEP = 2.0 ** -24


def up(v, m):
    return (v + m - 1) // m * m


def bf16(x):
    """Nearest BF16 (ties to even) of finite 64-bit values, as 64-bit values."""
    with np.errstate(over="ignore"):
        u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    u = (u + np.uint32(0x7FFF) + ((u >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xFFFF0000)
    return u.view(np.float32).astype(np.float64)


def _byte_values(kind):
    """The value of every byte of the 8-bit type."""
    bits, bias = (3, 7) if kind == E4M3 else (2, 15)
    out = np.empty(256)
    for i in range(256):
        e, m = (i & 0x7F) >> bits, i & ((1 << bits) - 1)
        v = m * 2.0 ** (1 - bias - bits) if e == 0 else (1 + m / (1 << bits)) * 2.0 ** (e - bias)
        if kind == E4M3 and (i & 0x7F) == 0x7F:
            v = np.nan
        if kind == E5M2 and e == 31:
            v = np.inf if m == 0 else np.nan
        out[i] = -v if i & 0x80 else v
    return out


VALUES = {E4M3: _byte_values(E4M3), E5M2: _byte_values(E5M2)}
LARGEST = {E4M3: 448.0, E5M2: 57344.0}


def to_bytes(v, kind):
    """Nearest byte of every |v| <= the type's largest, ties to the even byte; NaN gives a NaN byte, an
    infinity an infinity (or NaN)."""
    pos = VALUES[kind][:128]
    fin = pos[np.isfinite(pos)]
    a = np.abs(v)
    ok = np.isfinite(a)
    x = np.where(ok, a, 0.0)
    hi = np.minimum(np.searchsorted(fin, x), len(fin) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = x - fin[lo], fin[hi] - x
    take_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    b = np.where(take_hi, hi, lo)
    b = np.where(ok, b, 0x7F if kind == E4M3 else np.where(np.isinf(a), 0x7C, 0x7F))
    return (b | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def scale_bytes(amax, kind):
    """Smallest b >= 0 with amax <= largest * 2^(b - 127); 0 for 0."""
    out = np.zeros(amax.shape, dtype=np.int64)
    for b in range(247, -1, -1):
        out = np.where(amax <= LARGEST[kind] * 2.0 ** (b - 127), b, out)
    return out


def quantize(x, kind, block_rows=1):
    """(bytes, scale bytes) of blocks of block_rows x 128, in the C ABI's layout."""
    m, k = x.shape
    mp, kp = up(m, block_rows), up(k, BLOCK)
    t = np.zeros((mp, kp))
    t[:m, :k] = x
    t = t.reshape(mp // block_rows, block_rows, kp // BLOCK, BLOCK)
    finite = np.where(np.isfinite(t), np.abs(t), 0.0)
    b = scale_bytes(finite.max(axis=(1, 3)), kind)
    q = to_bytes(t / 2.0 ** (b - 127.0)[:, None, :, None], kind).reshape(mp, kp)[:m]
    s = np.zeros((mp // block_rows, up(kp // BLOCK, 4)), dtype=np.uint8)
    s[:, :kp // BLOCK] = b
    return q, s


def values(q, s, kind, cols, block_rows=1):
    """What the bytes stand for."""
    m, kp = q.shape
    e = np.repeat(np.repeat(s[:, :kp // BLOCK].astype(np.float64) - 127, block_rows, axis=0)[:m], BLOCK, axis=1)
    return (VALUES[kind][q] * 2.0 ** e)[:, :cols]


def spans(offsets, groups, rows):
    """Rows of every group: offsets clamped to 0..rows and to ascending order."""
    if offsets is None:
        return [(0, rows)]
    o = np.maximum.accumulate(np.clip(np.asarray(offsets, dtype=np.int64), 0, rows))
    return [(int(o[g]), int(o[g + 1])) for g in range(groups)]


def quantize_t(x, kind, groups, offsets, padded):
    """Transposed blocks along the tokens; columns of no group are 0 (and not to be compared)."""
    m, k = x.shape
    q = np.zeros((k, padded), dtype=np.uint8)
    s = np.zeros((k, up(padded // BLOCK, 4)), dtype=np.uint8)
    at = 0
    for a, b in spans(offsets, groups, m):
        if a == b:
            continue
        gq, gs = quantize(np.ascontiguousarray(x[a:b].T), kind)
        n = gq.shape[1]
        q[:, at:at + n] = gq
        s[:, at // BLOCK:(at + n) // BLOCK] = gs[:, :n // BLOCK]
        at += n
    return q, s, at


def route(logits, bias, cfg):
    """(ids, weights, scores) of 64-bit logits; cfg: a zc_route_config."""
    t, e = logits.shape
    with np.errstate(all="ignore"):
        if cfg.score == 1:
            s = 1.0 / (1.0 + np.exp(-logits))
        else:
            m = logits.max(axis=1, keepdims=True)
            p = np.exp(logits - np.where(np.isneginf(m), 0.0, m))
            total = p.sum(axis=1, keepdims=True)
            s = np.where(total == 0, 0.0, p / np.where(total == 0, 1.0, total))
        c = s + (0.0 if bias is None else bias[None])
        c = np.where(np.isnan(c), -np.inf, c)
        per = e // cfg.groups
        allowed = np.ones((t, e), dtype=bool)
        if cfg.groups > 1:
            g = -np.sort(-c.reshape(t, cfg.groups, per), axis=2)[:, :, :cfg.group_score].sum(axis=2)
            order = np.argsort(-g, axis=1, kind="stable")[:, :cfg.group_top]
            keep = np.zeros((t, cfg.groups), dtype=bool)
            np.put_along_axis(keep, order, True, axis=1)
            allowed = np.repeat(keep, per, axis=1)
        # experts outside the kept groups come after all others, whatever their score
        ids = np.empty((t, cfg.top_k), dtype=np.int64)
        for i in range(t):
            ids[i] = np.lexsort((np.arange(e), -c[i], ~allowed[i]))[:cfg.top_k]
        p = np.take_along_axis(s, ids, axis=1)
        w = p / (p.sum(axis=1, keepdims=True) + 1e-20) if cfg.renormalise else p
    return ids, w * float(np.float32(cfg.scale)), s


def route_backward(logits, cfg, ids, dw):
    """Gradient of the logits (64 bits) and the size of its terms, for tolerances."""
    zero_bias = None
    _, _, s = route(logits, zero_bias, cfg)
    t, e = logits.shape
    p = np.take_along_axis(s, ids, axis=1)
    a = float(np.float32(cfg.scale))
    d, size = a * dw, np.abs(a * dw)
    if cfg.renormalise:
        total = p.sum(axis=1, keepdims=True) + 1e-20
        size = (size + (size * p).sum(axis=1, keepdims=True) / total) / total
        d = (d - (d * p).sum(axis=1, keepdims=True) / total) / total
    ds, sz = np.zeros((t, e)), np.zeros((t, e))
    np.put_along_axis(ds, ids, d, axis=1)
    np.put_along_axis(sz, ids, size, axis=1)
    if cfg.score == 1:
        with np.errstate(over="ignore"):
            rest = 1.0 / (1.0 + np.exp(logits))
        return ds * s * rest, sz * s * rest
    dot = (ds * s).sum(axis=1, keepdims=True)
    return s * (ds - dot), s * (sz + (sz * s).sum(axis=1, keepdims=True))


def swiglu(g, u):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def swiglu_backward(g, u, dh):
    """(dgate, dup, sizes of dgate's terms)."""
    with np.errstate(over="ignore"):
        s, rest = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
    return dh * u * s * (1 + g * rest), dh * g * s, np.abs(dh * u) * s * (1 + np.abs(g) * rest)
