"""GPU: routing by scores at the edges: the documented error of a weight, pair by pair, and rows with fewer experts that
may be chosen than are asked for.  u = 2^-24."""
import numpy as np
import pytest
import torch

from activation_paging_gb300 import inputs
from gpu_util import host, to_dev
from oracle import layer

pytestmark = pytest.mark.gpu

ap = pytest.importorskip("activation_paging_gb300")

U = 2.0 ** -24
TINY = 2.0 ** -120


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(8, 8), (64, 8), (256, 32)])
@pytest.mark.parametrize("level,width", [(0, 1), (0, 40), (-30, 5), (-50, 10), (-80, 1), (-80, 8), (30, 20)])
def test_weights_within_the_documented_error(score, renorm, E, k, level, width):
    """(2 d + E / 32 + 40) u, d the distance of a pair's logit from the row's largest (renorm: from the largest chosen;
    sigmoid without renorm: 0)."""
    T = 2000
    logits = (level + width * (inputs.rng(E + k, 7).random((T, E)) - 0.5)).astype(np.float32)
    idx, w = ap.route_scored(to_dev(logits), k, score, renorm=renorm, scale=1.0)
    i, we, _, _ = layer.route_scored(logits, k, score, renorm=renorm)
    assert np.array_equal(host(idx), i)
    l = np.take_along_axis(logits, i, 1).astype(np.float64)
    d = l.max(1, keepdims=True) - l
    if score == "sigmoid" and not renorm:
        d = 0.0
    assert np.all(np.abs(host(w).astype(np.float64) - we) <= (2 * d + E / 32 + 40) * U * np.abs(we) + TINY)


def short_rows(T, E, groups):
    """Logits with many experts masked: rows with fewer than k to choose from in their groups, and none at all."""
    logits = inputs.router_logits(E + 1, T, E)
    off = inputs.rng(E, 8).random((T, E)) < np.linspace(0.0, 0.95, T)[:, None]
    logits[off] = -np.inf
    logits[T // 2] = -np.inf
    return logits


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k,groups,top", [(8, 4, 4, 2), (60, 6, 5, 1), (60, 6, 1, 1), (256, 8, 16, 2)])
@pytest.mark.parametrize("masked_by", ["logits", "bias"])
def test_gradient_of_experts_chosen_for_want_of_others(score, renorm, E, k, groups, top, masked_by):
    """They have weight 0 whatever their logits, so no gradient, and are no part of the others' sums.  The bound is that of
    all gradients: (2 d + E / 32 + 50) u of the sum of magnitudes, d at most the row's spread."""
    T = 200
    bias = (inputs.rng(3, 2).standard_normal(E) * 0.05).astype(np.float32)
    if masked_by == "logits":
        logits = short_rows(T, E, groups)
    else:
        logits = inputs.router_logits(E + 1, T, E)
        bias[inputs.rng(4, 2).permutation(E)[: E - k // 2]] = -np.inf  # fewer than k experts are on at all
    idx, w = ap.route_scored(to_dev(logits), k, score, to_dev(bias), groups, top, 2, renorm, 2.5)
    i, _, _, eligible = layer.route_scored(logits, k, score, bias, groups, top, 2, renorm, 2.5)
    assert np.array_equal(host(idx), i) and not eligible.all()
    dw = inputs.rng(5, 2).standard_normal((T, k)).astype(np.float32)
    got = host(ap.route_scored_backward(to_dev(logits), idx, to_dev(dw), score, renorm, 2.5, w=w)).astype(np.float64)
    want = layer.route_scored_backward(logits, i, dw, score, renorm, 2.5, eligible)
    size = np.abs(layer.route_scored_backward(logits, i, np.abs(dw), score, renorm, 2.5, eligible))
    finite = np.where(np.isfinite(logits), logits, 0.0).astype(np.float64)
    spread = (finite.max(1) - finite.min(1))[:, None]
    top_of = np.abs(size).max(1, keepdims=True) + 2.5 * np.abs(dw).max(1, keepdims=True)
    some = np.isfinite(logits).any(1)
    assert np.all((np.abs(got - want) <= (2 * spread + E / 32 + 50) * U * top_of + TINY)[some])
    assert not got[~some].any()
    # a pair that does not count has none, not even where the formula for all pairs has one
    off = np.where(eligible, 0.0, np.take_along_axis(got, i, 1).astype(np.float64))
    if not (score == "softmax" and not renorm):
        assert not off.any()


def test_gradient_of_rows_that_hold_nan():
    logits = inputs.router_logits(1, 4, 16)
    logits[1, 9] = np.nan
    for score in ("sigmoid", "softmax"):
        idx, w = ap.route_scored(to_dev(logits), 4, score)
        d = host(ap.route_scored_backward(to_dev(logits), idx, torch.ones_like(w), score, w=w))
        assert np.isnan(d[1, :4]).all() and not np.isnan(d[[0, 2, 3]]).any()


def test_weights_of_the_gradient_are_checked():
    logits = torch.zeros(4, 8, device="cuda")
    idx, w = ap.route_scored(logits, 2)
    for bad in (w[:2], w.double(), w.cpu(), w.t().contiguous().t()):
        with pytest.raises(ValueError, match="w must"):
            ap.route_scored_backward(logits, idx, w, w=bad)


def test_gradient_with_weights_in_a_graph_and_in_place():
    logits = torch.from_numpy(short_rows(300, 64, 4)).cuda()
    idx, w = ap.route_scored(logits, 8, groups=4, top_groups=2)
    dw, d, graph = torch.randn_like(w), torch.empty_like(logits), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ap.route_scored(logits, 8, groups=4, top_groups=2, idx=idx, w=w)
        ap.route_scored_backward(logits, idx, dw, dlogits=d, w=w)
    logits.copy_(logits.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    i, we = ap.route_scored(logits, 8, groups=4, top_groups=2)
    assert torch.equal(i, idx) and torch.equal(we, w)
    same = logits.clone()
    ap.route_scored_backward(same, i, dw, dlogits=same, w=we)
    assert torch.equal(same, d) and bool(torch.isfinite(d).all())
