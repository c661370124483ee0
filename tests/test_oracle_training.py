"""Pins of the 64-bit plain forms of the training operators: closed forms,
identities, and gradients against differences of the functions themselves."""
import numpy as np
import pytest

import oracle
from activation_paging_gb300 import inputs
from oracle import training


def test_balance_routes_as_the_oracle_router():
    logits = inputs.router_logits(3, 50, 12)
    logits[:, 3] = logits[:, 7]  # ties go to the lower id
    idx, w = oracle.route_topk(logits, 4)
    r = training.route_balance(logits, 4, 1.0)
    assert np.array_equal(r["idx"], idx)
    np.testing.assert_allclose(r["w"], w, rtol=2.0 ** -22)


@pytest.mark.parametrize("G", [1, 4])
def test_balanced_router_has_loss_coef(G):
    """Equal counts of every expert: loss = coef whatever the probabilities, since sum_e prob = 1."""
    T, E = 32, 8
    logits = np.full((T, E), -3.0, np.float32)
    logits[np.arange(T), np.arange(T) % E] = 2.0
    r = training.route_balance(logits, 1, 0.25, T // G)
    assert np.all(r["counts"] == T // G // E)
    np.testing.assert_allclose(r["prob"].sum(1), 1.0, rtol=1e-14)
    np.testing.assert_allclose(r["loss"], 0.25, rtol=1e-14)


def test_collapsed_router_has_loss_coef_times_experts_times_probability():
    T, E = 16, 4
    logits = np.zeros((T, E), np.float32)
    logits[:, 2] = np.log(5.0)
    r = training.route_balance(logits, 1, 1.0)
    assert r["counts"].tolist() == [[0, 0, T, 0]]
    np.testing.assert_allclose(r["loss"], E * 5 / 8, rtol=1e-7)


def test_masked_and_empty_groups_add_nothing():
    logits = inputs.router_logits(5, 24, 6)
    mask = np.ones(24, bool)
    mask[5:8] = False
    mask[8:16] = False  # the second group has no token
    r = training.route_balance(logits, 2, 1.0, 8, mask)
    one = training.route_balance(logits[:5], 2, 1.0)
    assert np.array_equal(r["counts"][0], one["counts"][0])
    np.testing.assert_allclose(r["prob"][0], one["prob"][0], rtol=1e-14)
    assert not r["counts"][1].any() and not r["prob"][1].any() and not r["slope"][1].any()
    np.testing.assert_allclose(r["loss"], (one["loss"] + training.route_balance(logits[16:], 2, 1.0)["loss"]) / 3,
                               rtol=1e-14)


def test_router_gradient_matches_differences():
    """f(logits) = <dw, w> + dloss * loss with the chosen experts (and so the counts) held."""
    T, E, k, S = 13, 9, 3, 5
    x = inputs.router_logits(11, T, E).astype(np.float64)
    x[2, 4] = -np.inf  # an expert that token 2 must not choose
    mask = np.ones(T, bool)
    mask[[3, 9]] = False
    dw = inputs.rng(1, 9).standard_normal((T, k))
    r = training.route_balance(x, k, 0.3, S, mask)

    def f(y):
        p = training.softmax(y)
        sel = np.take_along_axis(p, r["idx"], 1)
        on = mask[:, None]
        return float((sel / sel.sum(1, keepdims=True) * dw).sum() + 1.7 * (p * r["slope"][np.arange(T) // S] * on).sum())

    d = training.route_backward(x, r["idx"], r["w"], dw, r["slope"], 1.7, S, mask)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            if np.isinf(x[t, e]):
                assert d[t, e] == 0
                continue
            a, b = x.copy(), x.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((f(a) - f(b)) / (2 * h) - d[t, e]) < 1e-8
    # the loss is sum p * slope: the slope is its derivative with the counts held
    np.testing.assert_allclose(r["loss"], (training.softmax(x) * mask[:, None] * r["slope"][np.arange(T) // S]).sum(),
                               rtol=1e-13)


def test_embedding_gradient_is_the_transpose_of_the_lookup():
    """<dout, embed(table)> = <embed_backward(dout), table> for any table, and padding leaves its row alone."""
    V, H, T = 17, 6, 40
    g = inputs.rng(2, 8)
    table, dout, ids = g.standard_normal((V, H)), g.standard_normal((T, H)), g.integers(0, V, T)
    out = training.embed(table, ids, 1.5)
    d, rows, _ = training.embed_backward(dout, ids, V, 1.5)
    np.testing.assert_allclose((dout * out).sum(), (d * table).sum(), rtol=1e-12)
    assert rows.sum() == T
    d2, _, _ = training.embed_backward(dout, ids, V, 1.5, padding_idx=int(ids[0]), dtable=np.ones((V, H)))
    assert np.all(d2[ids[0]] == 1)
    others = np.arange(V) != ids[0]
    np.testing.assert_allclose(d2[others] - 1, d[others], atol=1e-12)


def test_embedding_skips_ids_outside():
    table = np.arange(8.0).reshape(4, 2)
    assert np.array_equal(training.embed(table, [-1, 4, 2], 2.0), [[0, 0], [0, 0], [8, 10]])
    d, rows, _ = training.embed_backward(np.ones((3, 2)), [-1, 4, 2], 4, 2.0)
    assert rows.tolist() == [0, 0, 1, 0] and d.sum() == 4
