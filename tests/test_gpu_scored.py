"""GPU parity: routing by scores, its gradient and the bias's step, against their
64-bit plain forms.

Ids and counts are compared exactly: the choice is that of the real values.  The
bounds of the rest follow from the kernels' single-precision steps (u = 2^-24):

* a chosen score: the distance d to the row's or the chosen's largest logit
  rounds once (d u in the exponent), expf is within 2 ulp (4 u), 1 + e^l and the
  quotient round (the exponential counted twice): (d + 10) u; the sum of k <= 32
  scores has five additions of terms with that error, the softmax's sum of E
  terms by 2^x (2 d + 4 + E / 32 + 5) u weighted by their shares (whose mean d is
  at most ln E < 7); division and scale two more: (2 d + E / 32 + 2 * 10 + 20) u;
* the gradient: products of such scores and differences of dw: the same bound
  times the sum of the magnitudes of its terms, with 10 u more.
"""
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


def spread(logits):
    x = np.where(np.isfinite(logits), logits.astype(np.float64), 0.0)
    return np.minimum(x.max(1) - x.min(1), 110.0)[:, None] if x.size else np.zeros((x.shape[0], 1))


def check(logits, k, score="sigmoid", bias=None, groups=1, top_groups=1, best=2, renorm=True, scale=1.0, mask=None,
          stream=None):
    T, E = logits.shape
    counts = torch.full((E,), 3, dtype=torch.int32, device="cuda")
    idx, w = ap.route_scored(to_dev(logits), k, score, None if bias is None else to_dev(bias), groups, top_groups, best, renorm,
                             scale, None if mask is None else to_dev(mask), counts, stream=stream)
    torch.cuda.synchronize()
    i, we, n, _ = layer.route_scored(logits, k, score, bias, groups, top_groups, best, renorm, scale, mask)
    assert np.array_equal(host(idx), i)
    assert np.array_equal(host(counts) - 3, n)
    got = host(w).astype(np.float64)
    odd = np.isnan(we)
    assert np.array_equal(np.isnan(got), odd)
    bound = (2 * spread(logits) + E / 32 + 40) * U * np.abs(we) + TINY
    assert np.all((np.abs(got - we) <= bound) | odd)
    return idx, w


def bias_of(E, seed=5, scale=0.05):
    return (inputs.rng(seed, 9).standard_normal(E) * scale).astype(np.float32)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,top,best", [
    (1, 1, 1, 1, 1, 1),
    (1, 8, 8, 1, 1, 1),
    (3, 2, 1, 2, 1, 1),
    (257, 60, 6, 5, 2, 2),
    (100, 33, 5, 11, 4, 2),
    (64, 64, 32, 32, 20, 2),      # groups of two, as many as lanes
    (129, 128, 8, 1, 1, 2),
    (1000, 256, 8, 8, 4, 2),
    (77, 254, 9, 2, 1, 1),
    (33, 512, 12, 16, 3, 2),
    (65, 513, 7, 27, 9, 2),
    (40, 1024, 32, 32, 1, 2),
    (31, 1024, 8, 1, 1, 1),
    (90, 1000, 8, 8, 3, 1),
])
@pytest.mark.parametrize("with_bias,renorm", [(True, True), (False, False)])
def test_against_double(score, T, E, k, groups, top, best, with_bias, renorm):
    logits = inputs.router_logits(T + E, T, E)
    mask = (np.arange(T) % 3 != 1)
    check(logits, k, score, bias_of(E, scale=0.05 if score == "sigmoid" else 0.2 / E) if with_bias else None, groups, top, best,
          renorm, 2.5, mask)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E", [16, 60, 256, 1024])
@pytest.mark.parametrize("groups", [1, 4])
def test_choices_nearer_than_single_precision(score, E, groups):
    """Biases that lift every expert to almost the same choice: their order is decided by differences of about 1e-9."""
    row = inputs.router_logits(E, 1, E)[0]
    s = layer.sigmoid(row) if score == "sigmoid" else layer.softmax(row[None])[0]
    bias = (0.75 - s).astype(np.float32)
    T = 50
    logits = np.repeat(row[None], T, 0)
    logits[1::2] += inputs.router_logits(3, T // 2, E) * 1e-7  # some rows a step off
    check(logits, min(8, E), score, bias, groups, max(1, groups // 2), 2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups", [(8, 2), (60, 1), (256, 8), (600, 6)])
@pytest.mark.parametrize("with_bias", [True, False])
def test_ties(score, E, groups, with_bias):
    """Equal logits and equal biases: the lower expert, the lower group."""
    T = 40
    logits = inputs.rng(4, 3).integers(-2, 3, (T, E)).astype(np.float32)
    logits[0] = 0.0
    bias = np.zeros(E, np.float32) if with_bias else None
    check(logits, min(6, E // groups), score, bias, groups, 1, 2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
def test_masked_experts_and_odd_rows(score, renorm, with_bias):
    T, E, k = 64, 60, 6
    logits = inputs.router_logits(11, T, E)
    logits[1] = -np.inf                          # nothing to choose
    logits[2, 3:] = -np.inf                      # fewer than k
    logits[3, ::2] = -np.inf
    logits[4, 7] = np.nan
    logits[5] = np.nan
    logits[6, 9] = np.inf
    logits[7] = np.finfo(np.float32).min         # the type's lowest value is a number
    logits[8, 5:] = np.finfo(np.float32).min
    logits[9] = -200.0 - np.arange(E)            # sigmoids below the smallest number
    logits[10] = 100.0 + np.arange(E) / 64       # sigmoids of 1 in single precision, and in double
    logits[11] = np.arange(E) - 30.0
    bias = None
    if with_bias:
        bias = bias_of(E)
        bias[5], bias[6], bias[8] = -np.inf, np.nan, -1e9
    for groups, top, best in ((1, 1, 1), (5, 2, 2), (5, 2, 1), (10, 2, 2)):
        check(logits, k, score, bias, groups, top, best, renorm, 1.0, (np.arange(T) % 2 == 0))


def test_offsets_of_rows():
    """Rows that do not begin on 16-byte boundaries, and a bias that does not."""
    base = to_dev(inputs.router_logits(2, 1, 50 * 128 + 1)[0])
    logits = base[1:].view(50, 128)
    b = to_dev(bias_of(130))
    a = ap.route_scored(logits, 8, bias=b[1:129], groups=4, top_groups=2)
    c = ap.route_scored(logits.clone(), 8, bias=b[1:129].clone(), groups=4, top_groups=2)
    assert all(torch.equal(x, y) for x, y in zip(a, c))


def test_softmax_routing_is_route_topk():
    logits = inputs.router_logits(8, 500, 128)
    a = ap.route_topk(to_dev(logits), 8)
    b = ap.route_scored(to_dev(logits), 8, score="softmax")
    assert torch.equal(a[0], b[0])
    assert torch.allclose(a[1], b[1], rtol=2 ** -20, atol=0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 8), (257, 60, 6), (100, 128, 8), (64, 256, 8), (33, 511, 32), (20, 1024, 9)])
def test_gradient(score, renorm, T, E, k):
    logits = inputs.router_logits(T, T, E)
    if T > 4 and E > 8:
        logits[2, ::3] = -np.inf
        logits[3] -= 300.0 if score == "sigmoid" else 0.0
    idx, _, _, _ = layer.route_scored(logits, k, score)
    dw = inputs.rng(T, 6).standard_normal((T, k)).astype(np.float32)
    got = host(ap.route_scored_backward(to_dev(logits), to_dev(idx), to_dev(dw), score, renorm, 2.5)).astype(np.float64)
    e = layer.route_scored_backward(logits, idx, dw, score, renorm, 2.5)
    # magnitudes: the same formula with |dw| and its mean added instead of subtracted
    size = np.abs(layer.route_scored_backward(logits, idx, np.abs(dw), score, renorm, 2.5))
    top = np.abs(dw).max(1, keepdims=True) * 2.5
    p = np.maximum(layer.softmax(logits) if score == "softmax" and not renorm else (e != 0) * 1.0, 0)
    bound = (2 * spread(logits) + E / 32 + 50) * U * np.maximum(2 * top * p, size) + TINY
    assert np.all(np.abs(got - e) <= bound)
    same = to_dev(logits)
    ap.route_scored_backward(same, to_dev(idx), to_dev(dw), score, renorm, 2.5, dlogits=same)  # in place
    assert np.array_equal(host(same).astype(np.float64), got)


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
def test_gradient_against_differences(score, renorm):
    T, E, k, h = 6, 24, 4, 1e-6
    x = inputs.router_logits(1, T, E)
    idx, _, _, _ = layer.route_scored(x, k, score)
    dw = inputs.rng(2, 6).standard_normal((T, k)).astype(np.float32)
    got = host(ap.route_scored_backward(to_dev(x), to_dev(idx), to_dev(dw), score, renorm, 1.5))

    def weights(v):
        s = layer.sigmoid(v) if score == "sigmoid" else layer.softmax(v)
        w = np.take_along_axis(s, idx.astype(np.int64), 1)
        return 1.5 * (w / w.sum(1, keepdims=True) if renorm else w)
    for e in range(E):
        up, down = x.astype(np.float64), x.astype(np.float64)
        up[:, e] += h
        down[:, e] -= h
        diff = ((weights(up) - weights(down)) * dw).sum(1) / (2 * h)
        # differences: h^2 of the third derivative (below 1e-11), and 2^-52 / h of the values
        assert np.all(np.abs(got[:, e] - diff) <= 2e-6 * (1 + np.abs(dw).sum(1)))


def test_bad_ids_of_the_gradient():
    T, E, k = 10, 16, 3
    logits = inputs.router_logits(1, T, E)
    idx, _, _, _ = layer.route_scored(logits, k)
    idx[4, 1], idx[6, 0] = -1, E
    dw = inputs.rng(2, 6).standard_normal((T, k)).astype(np.float32)
    for score, renorm in (("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = ap.route_scored_backward(to_dev(logits), to_dev(idx), to_dev(dw), score, renorm, status=status)
        e = layer.route_scored_backward(logits, idx, dw, score, renorm)
        assert np.all(np.abs(host(got) - e) <= 100 * U * (np.abs(dw).max() + 1))
        assert int(status) == ap.FLAG_BAD_INDEX


def test_bias_step():
    for E in (1, 5, 64, 1000, 1024):
        counts = inputs.rng(E, 2).integers(0, 9, E).astype(np.int32)
        counts[0] = 2 ** 31 - 1 if E == 1000 else counts[0]
        bias = bias_of(E)
        for reset in (False, True):
            b, c = to_dev(bias), to_dev(counts)
            ap.route_bias_step(b, c, 1e-3, reset=reset)
            assert np.array_equal(host(b), layer.route_bias_step(bias, counts, 1e-3))
            assert np.array_equal(host(c), counts * (not reset))


def test_captured_and_replayed_with_new_logits():
    T, E, k = 300, 256, 8
    logits, bias = to_dev(inputs.router_logits(1, T, E)), to_dev(bias_of(E))
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    dw = torch.randn(T, k, device="cuda")
    d = torch.empty(T, E, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ap.route_scored(logits, k, bias=bias, groups=8, top_groups=4, counts=counts, idx=idx, w=w)
        ap.route_scored_backward(logits, idx, dw, dlogits=d)
        ap.route_bias_step(bias, counts, 1e-2, reset=True)
    b = bias_of(E)
    for r in range(3):
        new = inputs.router_logits(20 + r, T, E)
        logits.copy_(to_dev(new))
        g.replay()
        torch.cuda.synchronize()
        i, _, n, _ = layer.route_scored(new, k, bias=b, groups=8, top_groups=4)
        assert np.array_equal(host(idx), i)
        b = layer.route_bias_step(b, n, 1e-2)
        assert np.array_equal(host(bias), b)
        assert np.all(np.abs(host(d) - layer.route_scored_backward(new, i, host(dw))) <= 1e-5)
        assert not counts.any()


def test_empty_batch():
    idx, w = ap.route_scored(torch.empty(0, 8, device="cuda"), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    assert ap.route_scored_backward(torch.empty(0, 8, device="cuda"), idx, w).shape == (0, 8)


def test_refusals():
    logits = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError, match="score"):
        ap.route_scored(logits, 2, score="relu")
    with pytest.raises(ValueError, match="bias"):
        ap.route_scored(logits, 2, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError, match="counts"):
        ap.route_scored(logits, 2, counts=torch.zeros(8, device="cuda"))
    with pytest.raises(ValueError, match="idx"):
        ap.route_scored(logits, 2, idx=torch.zeros(4, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ap.APError, match="groups"):
        ap.route_scored(logits, 5, groups=4, top_groups=2)
    with pytest.raises(ap.APError, match="groups"):
        ap.route_scored(logits, 2, groups=3)
    with pytest.raises(ValueError, match="dw"):
        ap.route_scored_backward(logits, torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda"))
