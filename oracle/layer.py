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


def route_scored_backward(logits, idx, dw, score="sigmoid", renorm=True, scale=1.0):
    T, E = logits.shape
    x, dw = logits.astype(np.float64), dw.astype(np.float64)
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
