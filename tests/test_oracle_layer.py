"""Pins of the 64-bit plain forms of routing by scores, the experts' products and
the weights' update: hand-made cases, identities, and gradients and steps against
torch's own in double precision."""
import numpy as np
import pytest
import torch

from activation_paging_gb300 import inputs
from oracle import layer, training


def test_scored_routing_by_hand():
    logits = np.array([[0.0, 3.0, 1.0, 2.0, -1.0, 2.0, 0.0, 5.0]], np.float32)
    # groups of two: sums of both sigmoids; (0, 3) 1.45, (1, 2) 1.61, (-1, 2) 1.15, (0, 5) 1.49
    idx, w, n, _ = layer.route_scored(logits, 2, groups=4, top_groups=2)
    assert idx.tolist() == [[7, 3]] and n.tolist() == [0, 0, 0, 1, 0, 0, 0, 1]
    s = 1 / (1 + np.exp(-np.array([5.0, 2.0])))
    np.testing.assert_allclose(w[0], s / s.sum(), rtol=1e-14)
    idx, w, _, _ = layer.route_scored(logits, 2, groups=4, top_groups=1, best=1, renorm=False, scale=2.0)
    assert idx.tolist() == [[7, 6]]
    np.testing.assert_allclose(w[0], [2 / (1 + np.exp(-5.0)), 1.0], rtol=1e-14)
    bias = np.zeros(8, np.float32)
    bias[4] = 10.0  # the bias chooses, but is no part of the weight
    idx, w, _, _ = layer.route_scored(logits, 1, bias=bias, renorm=False)
    assert idx.tolist() == [[4]]
    np.testing.assert_allclose(w[0], [1 / (1 + np.exp(1.0))], rtol=1e-14)


def test_softmax_scores_are_the_balance_routers():
    logits = inputs.router_logits(3, 40, 12)
    a, b = layer.route_scored(logits, 4, "softmax"), training.route_balance(logits, 4, 1.0)
    assert np.array_equal(a[0], b["idx"]) and np.array_equal(a[2], b["counts"][0])
    np.testing.assert_allclose(a[1], b["w"], rtol=1e-12)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_scored_gradient_is_autograd(score, renorm):
    x = torch.tensor(inputs.router_logits(1, 20, 9), dtype=torch.float64, requires_grad=True)
    idx, w, _, _ = layer.route_scored(x.detach().numpy().astype(np.float32), 3, score, renorm=renorm, scale=1.5)
    dw = np.random.default_rng(0).standard_normal((20, 3))
    s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    v = s.gather(1, torch.from_numpy(idx).long())
    v = 1.5 * (v / v.sum(1, keepdim=True) if renorm else v)
    np.testing.assert_allclose(v.detach().numpy(), w, rtol=1e-6)
    (v * torch.from_numpy(dw)).sum().backward()
    np.testing.assert_allclose(layer.route_scored_backward(x.detach().numpy(), idx, dw, score, renorm, 1.5), x.grad.numpy(),
                               rtol=1e-10, atol=1e-13)


def test_bias_step_moves_towards_the_mean():
    b = layer.route_bias_step(np.zeros(4, np.float32), np.array([1, 3, 2, 2], np.int32), 0.5)
    assert b.tolist() == [0.5, -0.5, 0.0, 0.0]


@pytest.mark.parametrize("kind", [None, "silu", "gelu", "swiglu"])
def test_expert_products_are_autograds(kind):
    g = np.random.default_rng(2)
    seg, live = np.array([3, 0, 9], np.int32), np.array([5, 3, 0], np.int32)
    wide = 14 if kind == "swiglu" else 7
    x, W, b = g.standard_normal((12, 6)), g.standard_normal((3, wide, 6)), g.standard_normal((3, wide))
    res, dy, V = g.standard_normal((12, 7)), g.standard_normal((12, 4)), g.standard_normal((3, 4, 7))
    z, out, _ = layer.expert_linear(x, W, seg, live, b, kind, res)
    tx, tW, tb = (torch.tensor(t, requires_grad=True) for t in (x, W, b))
    fn = {None: lambda t: t, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
          "swiglu": lambda t: torch.nn.functional.silu(t[:, :7]) * t[:, 7:]}[kind]
    loss = 0
    for e, at in ((0, slice(3, 8)), (1, slice(0, 3))):
        tz = tx[at] @ tW[e].t() + tb[e]
        h = fn(tz)
        np.testing.assert_allclose(out[at], (h + torch.from_numpy(res[at])).detach().numpy(), rtol=1e-12)
        loss = loss + ((h @ torch.from_numpy(V[e]).t()) * torch.from_numpy(dy[at])).sum()
    loss.backward()
    assert np.isnan(out[8:]).all()
    dz, _ = layer.expert_linear_dx(dy, V, seg, live, kind, z)
    dW, db, _, _ = layer.expert_linear_dw(np.nan_to_num(dz), x, seg, live, 3)
    dx, _ = layer.expert_linear_dx(np.nan_to_num(dz), W, seg, live)
    np.testing.assert_allclose(dW, tW.grad.numpy(), rtol=1e-9, atol=1e-11)
    np.testing.assert_allclose(db, tb.grad.numpy(), rtol=1e-9, atol=1e-11)
    np.testing.assert_allclose(dx[:8], tx.grad.numpy()[:8], rtol=1e-9, atol=1e-11)


def test_adamw_is_torchs():
    g = torch.Generator().manual_seed(1)
    p = torch.nn.Parameter(torch.randn(50, generator=g, dtype=torch.float64))
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.95), eps=1e-6, weight_decay=0.1)
    mine, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        p.grad = torch.randn(50, generator=g, dtype=torch.float64)
        mine, m, v, _ = layer.adamw_step(mine, p.grad.numpy(), m, v, t, 1e-2, (0.9, 0.95), 1e-6, 0.1)
        opt.step()
        np.testing.assert_allclose(mine, p.detach().numpy(), rtol=1e-12)


def test_noise_is_even_and_reproducible():
    low, high = layer.adamw_noise(5, 3, 2, 1 << 16)
    for u in (low, high):
        assert 0 <= u.min() and u.max() < 1
        # the mean of 65536 even fractions has a deviation of 0.29 / 256
        assert abs(u.mean() - 0.5) < 5 * 0.29 / 256
    assert abs(np.corrcoef(low, high)[0, 1]) < 5 / 256
    again = layer.adamw_noise(5, 3, 2, 100)
    assert np.array_equal(again[0], low[:100])
    assert not np.array_equal(layer.adamw_noise(5, 4, 2, 100)[0], low[:100])
    assert not np.array_equal(layer.adamw_noise(5, 3, 3, 100)[0], low[:100])


def test_codes_by_hand():
    m, v = layer.adamw_decode(np.array([-127, 0, 10], np.int8), np.array([255, 1, 0], np.uint8), np.array([2.0], np.float32),
                              np.array([0.5], np.float32))
    assert m.tolist() == [-2.0 * 127 ** 2, 0.0, 200.0] and v.tolist() == [(0.5 * 255 ** 2) ** 2, 0.25, 0.0]
