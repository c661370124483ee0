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
