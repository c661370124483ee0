"""64-bit plain forms of the training operators: routing with a balance loss,
the router's gradient, the embedding lookup and its gradient.

Written from the formulas in double precision numpy, with no code of the
package: they say what the operators compute, not how."""
from __future__ import annotations

import numpy as np


def _groups(T: int, group_tokens: int):
    S = group_tokens if 0 < group_tokens < T else max(T, 1)
    return S, -(-T // S)


def softmax(logits: np.ndarray) -> np.ndarray:
    """Rows of probabilities; a row of -infinity alone has none (zeros)."""
    x = logits.astype(np.float64)
    top = x.max(1, keepdims=True) if x.size else x[:, :1]
    live = np.isfinite(top)
    z = np.where(live, np.exp(x - np.where(live, top, 0.0)), 0.0)
    s = z.sum(1, keepdims=True)
    return np.divide(z, s, out=np.zeros_like(z), where=s > 0)


def counting(logits: np.ndarray, mask) -> np.ndarray:
    """Tokens that count: unmasked, with a logit above -infinity."""
    on = np.ones(logits.shape[0], bool) if mask is None else np.asarray(mask).astype(bool)
    some = np.zeros(logits.shape[0], bool)
    some[on] = logits[on].max(1) > -np.inf if on.any() else False
    return on & some


def route_balance(logits, k, coef, group_tokens=0, mask=None):
    """idx, w, counts, prob, slope, loss (w, prob, slope, loss in 64 bits)."""
    T, E = logits.shape
    S, G = _groups(T, group_tokens)
    on = counting(logits, mask)
    idx = np.argsort(-logits.astype(np.float64), axis=1, kind="stable")[:, :k].astype(np.int32)
    p = softmax(logits)
    sel = np.take_along_axis(p, idx, 1)
    total = sel.sum(1, keepdims=True)
    w = np.divide(sel, total, out=np.zeros_like(sel), where=total > 0)
    counts = np.zeros((G, E), np.int32)
    prob, slope, loss = np.zeros((G, E)), np.zeros((G, E)), 0.0
    for g in range(G):
        m = np.flatnonzero(on[g * S:(g + 1) * S]) + g * S
        if not m.size:
            continue
        np.add.at(counts[g], idx[m].ravel(), 1)
        prob[g] = p[m].sum(0) / m.size
        slope[g] = coef * E * counts[g] / (G * k * float(m.size) ** 2)
        loss += coef / G * E * float((counts[g] / (m.size * k) * prob[g]).sum())
    return {"idx": idx, "w": w, "counts": counts, "prob": prob, "slope": slope, "loss": loss}


def route_backward(logits, idx=None, w=None, dw=None, slope=None, dloss=1.0, group_tokens=0, mask=None):
    T, E = logits.shape
    S, _ = _groups(T, group_tokens)
    d = np.zeros((T, E))
    if slope is not None:
        on = counting(logits, mask)
        p = softmax(logits[on])
        s = slope.astype(np.float64)[np.arange(T) // S][on]
        d[on] = dloss * p * (s - (p * s).sum(1, keepdims=True))
    if dw is not None:
        w, dw = w.astype(np.float64), dw.astype(np.float64)
        dz = w * (dw - (w * dw).sum(1, keepdims=True))
        for j in range(idx.shape[1]):
            ok = (idx[:, j] >= 0) & (idx[:, j] < E)
            d[np.flatnonzero(ok), idx[ok, j]] += dz[ok, j]
    return d


def embed(table, ids, scale):
    ids = np.asarray(ids, np.int64)
    ok = (ids >= 0) & (ids < table.shape[0])
    out = np.zeros((ids.size, table.shape[1]))
    out[ok] = table.astype(np.float64)[ids[ok]] * scale
    return out


def embed_backward(dout, ids, V, scale, padding_idx=-1, dtable=None):
    """The gradient, and (for error bounds) each id's rows and the sum of their magnitudes."""
    ids = np.asarray(ids, np.int64)
    ok = (ids >= 0) & (ids < V) & (ids != padding_idx)
    g = dout.astype(np.float64)[ok]
    total, size, rows = np.zeros((V, dout.shape[1])), np.zeros((V, dout.shape[1])), np.zeros(V, np.int64)
    np.add.at(total, ids[ok], g)
    np.add.at(size, ids[ok], np.abs(g))
    np.add.at(rows, ids[ok], 1)
    out = scale * total
    if dtable is not None:
        out += dtable.astype(np.float64)
    return out, rows, size * abs(scale)
