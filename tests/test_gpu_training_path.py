"""The training operators in the layer that uses them: its gradients against
64-bit autograd, and the example's training run."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

pytest.importorskip("activation_paging_gb300")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def reference_gradients(layer, ids, target, mask, S, idx, weight):
    """The layer's loss (cross entropy + balance loss) in double precision, experts and counts held as chosen."""
    p = {n: v.double().requires_grad_() for n, v in layer.params.items()}
    T, E, k, G = ids.shape[0], layer.E, layer.k, ids.shape[0] // S
    m = mask.double()
    table = torch.where((torch.arange(layer.V, device=ids.device) == 0)[:, None], p["table"].detach(), p["table"])
    x = table[ids] * layer.scale
    prob = torch.softmax(x @ p["router"], 1)
    sel = prob.gather(1, idx.long())
    w = sel / sel.sum(1, keepdim=True)
    out = sum(w[:, j, None] * torch.einsum("th,tho->to", x, p["experts"][idx[:, j].long()]) for j in range(k))
    z = out @ p["head"]
    n = m.sum()
    ce = ((torch.logsumexp(z, 1) - z.gather(1, target[:, None])[:, 0]) * m).sum() / n
    ng = m.view(G, S).sum(1)
    chosen = torch.zeros(T, E, dtype=torch.float64, device=ids.device).scatter_(1, idx.long(), 1.0) * m[:, None]
    share = chosen.view(G, S, E).sum(1) / (ng * k)[:, None]
    mean = (prob * m[:, None]).view(G, S, E).sum(1) / ng[:, None]
    balance = layer.coef / G * E * (share * mean).sum()
    (weight * (ce + balance)).backward()
    return float(ce.detach()), float(balance.detach()), {n: v.grad for n, v in p.items()}


def test_layer_gradients_match_double_precision_autograd():
    """Every BF16 rounding (x, expert weights, y, out, dout, dy, dxd, dx: eight on the longest path) is relative 2^-8 at
    most of the value it rounds, so a gradient differs by at most about 8 x 2^-8 = 3.1% of its norm."""
    import train_moe_tokens as ex
    layer = ex.Layer(max_tokens=512, coef=0.5, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    follow = torch.arange(layer.V, device="cuda").roll(-1)
    follow[0], follow[-1] = 0, 1
    ids, target, mask = ex.batch(follow, 8, 64, g)
    s = layer.pool.stream
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = layer.step(ids, target, mask, 64, 0.5)
        x = layer.params["table"][ids] * layer.scale
        idx = torch.topk(x.bfloat16().float() @ layer.params["router"], layer.k, dim=1)[1]
    torch.cuda.synchronize()
    ce, balance, grads = reference_gradients(layer, ids, target, mask, 64, idx, 0.5)
    assert abs(float(got["loss"]) - ce) <= 8 * 2.0 ** -8 * ce
    assert abs(float(got["balance"]) - balance) <= 8 * 2.0 ** -8 * balance
    assert int(got["counts"].sum()) == int(mask.sum()) * layer.k
    for n, e in grads.items():
        err = float((layer.grads[n].double() - e).norm() / e.norm())
        assert err <= 8 * 2.0 ** -8, (n, err)
    assert not layer.grads["table"][0].any()  # the padding id


def test_example_learns():
    import train_moe_tokens as ex
    h = ex.train(steps=60)
    first, last = h[0], h[-1]
    assert first[0] > 4.5            # ln 256 = 5.5 before it has learnt anything
    assert last[0] < 0.5 * first[0]
    assert last[1] < 0.04            # coef = 0.02 when the experts share the tokens evenly
    assert max(last[2]) < 4 * sum(last[2]) / len(last[2])
