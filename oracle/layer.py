"""64-bit plain forms of routing by scores, the experts' products and the
weights' update.

Written from the formulas in double precision numpy, with no code of the
package: they say what the operators compute, not how."""
from __future__ import annotations

import numpy as np

from .training import softmax


def sigmoid(x: np.ndarray) -> np.ndarray:
    x = x.astype(np.float64)
    with np.errstate(over="ignore"):
        return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


def _stable_top(c: np.ndarray, k: int) -> np.ndarray:
    return np.argsort(-c, axis=1, kind="stable")[:, :k]


def route_scored(logits, k, score="sigmoid", bias=None, groups=1, top_groups=1, best=2, renorm=True, scale=1.0, mask=None):
    """idx, w (64 bits), counts, and which chosen experts may be chosen at all."""
    T, E = logits.shape
    x = logits.astype(np.float64)
    odd = np.isnan(x).any(1) if score == "sigmoid" else (np.isnan(x) | (x == np.inf)).any(1)
    clean = np.where(odd[:, None], 0.0, x)
    s = sigmoid(clean) if score == "sigmoid" else softmax(clean)
    # scores rise with the logits: where only their order counts, it is taken from these, which 64 bits tell apart
    # where they no longer do the scores (sigmoids of 40 and 41)
    c = clean if bias is None and (groups == 1 or best == 1) else s + (0.0 if bias is None else bias.astype(np.float64))
    c = np.where(np.isnan(c) | (x == -np.inf) | odd[:, None], -np.inf, c)
    if groups > 1:
        size = E // groups
        by = -np.sort(-c.reshape(T, groups, size), axis=2)[:, :, : best]
        by = by[:, :, 0] if best == 1 else by[:, :, 0] + by[:, :, 1]
        keep = np.zeros((T, groups), bool)
        np.put_along_axis(keep, _stable_top(by, top_groups), True, 1)
        c = np.where(np.repeat(keep, size, 1), c, -np.inf)
    idx = _stable_top(c, k)
    eligible = np.take_along_axis(c, idx, 1) > -np.inf
    if renorm:
        # shares of the chosen scores, whatever their size: from their logarithms
        l = np.take_along_axis(clean, idx, 1)
        logs = l if score == "softmax" else -np.logaddexp(0.0, -l)
        w = softmax(np.where(eligible, logs, -np.inf))
    else:
        w = np.where(eligible, np.take_along_axis(s, idx, 1), 0.0)
    w = w * scale
    w[odd] = np.nan
    some = odd | (x.max(1, initial=-np.inf) > -np.inf)
    on = some if mask is None else some & np.asarray(mask).astype(bool)
    counts = np.bincount(idx[on].ravel(), minlength=E)
    return idx.astype(np.int32), w, counts.astype(np.int32), eligible


def route_scored_backward(logits, idx, dw, score="sigmoid", renorm=True, scale=1.0, eligible=None):
    """eligible: the pairs that count (route_scored's last result); all without it."""
    T, E = logits.shape
    x, dw = logits.astype(np.float64), dw.astype(np.float64)
    if eligible is not None:
        idx = np.where(eligible, idx, -1)
    d = np.zeros((T, E))
    ok = (idx >= 0) & (idx < E)
    at = np.where(ok, idx, 0).astype(np.int64)
    l = np.where(ok, np.take_along_axis(x, at, 1), -np.inf)
    if score == "softmax" and not renorm:
        p = softmax(x)
        g = np.zeros((T, E))
        np.add.at(g, (np.arange(T)[:, None], at), np.where(ok, scale * dw, 0.0))
        return p * (g - (p * g).sum(1, keepdims=True))
    if renorm:
        r = softmax(l if score == "softmax" else np.where(ok & (l > -np.inf), -np.logaddexp(0.0, -np.where(ok & (l > -np.inf), l, 0.0)), -np.inf))
        part = r * (dw - (r * dw).sum(1, keepdims=True))
        if score == "sigmoid":
            part = part * sigmoid(-np.where(l > -np.inf, l, 0.0))
    else:
        part = np.where(l > -np.inf, sigmoid(l) * sigmoid(-l), 0.0) * dw
    np.add.at(d, (np.arange(T)[:, None], at), np.where(ok, scale * part, 0.0))
    return d


def route_bias_step(bias, counts, rate):
    n = counts.astype(np.int64)
    return (bias + np.float32(rate) * np.sign(n.sum() - n.size * n).astype(np.float32)).astype(np.float32)


# ---- the weights' update ---------------------------------------------------------

BLOCK = 256


def _mix(x):
    x = (x ^ (x >> 16)) * 0x85EBCA6B & 0xFFFFFFFF
    x = (x ^ (x >> 13)) * 0xC2B2AE35 & 0xFFFFFFFF
    return x ^ (x >> 16)


def adamw_noise(seed: int, t: int, tensor: int, n: int):
    """The low and high 16 bits, as fractions, that round the codes of m and v."""
    key = _mix((tensor + _mix((seed + 0x9E3779B9 * t) & 0xFFFFFFFF)) & 0xFFFFFFFF)
    e = np.arange(n, dtype=np.uint64) * np.uint64(0x9E3779B9)
    x = (e + np.uint64(key)) & np.uint64(0xFFFFFFFF)
    m32 = np.uint64(0xFFFFFFFF)
    x = (x ^ (x >> np.uint64(16))) * np.uint64(0x85EBCA6B) & m32
    x = (x ^ (x >> np.uint64(13))) * np.uint64(0xC2B2AE35) & m32
    x = (x ^ (x >> np.uint64(16))).astype(np.int64)
    return (x & 0xFFFF) / 65536.0, (x >> 16) / 65536.0


def adamw_decode(cm, cv, sm, sv):
    """(m, v) of codes and scales."""
    n = cm.size
    each = lambda s: np.repeat(s.astype(np.float64), BLOCK)[:n]  # noqa: E731
    c, r = cm.astype(np.float64), cv.astype(np.float64) ** 2 * each(sv)
    return c * np.abs(c) * each(sm), r * r


def adamw_codes(x, r, top, power, rounding="codes"):
    """Codes of magnitudes x in units of their scale (sqrt(v)'s too), with the fractions r; power: of the values that
    count, 1 for m, 2 for v."""
    c = np.floor(np.sqrt(x))
    if rounding == "codes":
        return np.minimum(np.floor(np.sqrt(x) + r), top)
    low, high = c ** (2 * power), (c + 1) ** (2 * power)
    return np.minimum(c + ((r + 0.5 / 65536) * (high - low) < x ** power - low), top)


def block_max(x):
    pad = np.zeros(-(-x.size // BLOCK) * BLOCK)
    pad[:x.size] = np.abs(x)
    return pad.reshape(-1, BLOCK).max(1)


def adamw_step(p, g, m, v, t, lr, betas, eps, weight_decay, scale=1.0):
    """(p, m, v, the step's change) after step t, in 64 bits, from 64-bit moments."""
    g = g.astype(np.float64) * scale
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    change = lr * (m / (1 - betas[0] ** t)) / (np.sqrt(v / (1 - betas[1] ** t)) + eps)
    return p.astype(np.float64) * (1 - lr * weight_decay) - change, m, v, change


# ---- the experts' products ---------------------------------------------------------

def _cdf(z):
    from math import erfc, sqrt
    return 0.5 * np.vectorize(erfc, otypes=[np.float64])(-z / sqrt(2.0)) if z.size else z


def act(kind, z):
    """act(z); swiglu: of the halves of z's columns."""
    if kind == "swiglu":
        n = z.shape[1] // 2
        return z[:, :n] * sigmoid(z[:, :n]) * z[:, n:]
    return z * sigmoid(z) if kind == "silu" else z * _cdf(z) if kind == "gelu" else z


def act_backward(kind, z, d):
    """d act(z) / dz times d."""
    if kind is None:
        return d
    if kind == "gelu":
        return d * (_cdf(z) + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi))
    n = d.shape[1]
    g = z[:, :n]
    s = sigmoid(g)
    slope = s * (1.0 + g * (1.0 - s))
    return d * slope if kind == "silu" else np.concatenate([d * z[:, n:] * slope, d * g * s], 1)


def expert_rows(seg, live, rows):
    """(expert, its rows) of every valid segment."""
    for e, (a, n) in enumerate(zip(seg.tolist(), live.tolist())):
        if a >= 0 and n > 0 and a + n <= rows:
            yield e, slice(a, a + n)


def expert_linear(x, W, seg, live, bias=None, kind=None, residual=None):
    """(z, out, and for error bounds the sums of magnitudes of z's terms): NaN in rows of no expert."""
    wide = W.shape[1]
    z, size = np.full((x.shape[0], wide), np.nan), np.zeros((x.shape[0], wide))
    for e, at in expert_rows(seg, live, x.shape[0]):
        b = 0.0 if bias is None else bias[e].astype(np.float64)
        z[at] = x[at] @ W[e].T + b
        size[at] = np.abs(x[at]) @ np.abs(W[e]).T + np.abs(b)
    out = np.full((x.shape[0], wide // 2 if kind == "swiglu" else wide), np.nan)
    for e, at in expert_rows(seg, live, x.shape[0]):
        out[at] = act(kind, z[at]) + (0.0 if residual is None else residual[at])
    return z, out, size


def expert_linear_dx(dy, W, seg, live, kind=None, pre=None, residual=None):
    """(dx, sums of magnitudes before the activation's slope)"""
    cols = W.shape[2]
    dx = np.full((dy.shape[0], 2 * cols if kind == "swiglu" else cols), np.nan)
    size = np.zeros((dy.shape[0], cols))
    for e, at in expert_rows(seg, live, dy.shape[0]):
        d = dy[at] @ W[e] + (0.0 if residual is None else residual[at])
        size[at] = np.abs(dy[at]) @ np.abs(W[e]) + (0.0 if residual is None else np.abs(residual[at]))
        dx[at] = act_backward(kind, None if kind is None else pre[at], d)
    return dx, size


def expert_linear_dw(dy, x, seg, live, E):
    """(dW, dbias, sums of magnitudes of both)"""
    dW, db = np.zeros((E, dy.shape[1], x.shape[1])), np.zeros((E, dy.shape[1]))
    sW, sb = np.zeros_like(dW), np.zeros_like(db)
    for e, at in expert_rows(seg, live, x.shape[0]):
        dW[e], db[e] = dy[at].T @ x[at], dy[at].sum(0)
        sW[e], sb[e] = np.abs(dy[at]).T @ np.abs(x[at]), np.abs(dy[at]).sum(0)
    return dW, db, sW, sb
