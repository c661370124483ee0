"""Routing by scores, the experts' products and the weights' update in the layer
that uses them: its gradients against 64-bit autograd, and the example's run."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ap = pytest.importorskip("activation_paging_gb300")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def reference(layer, ids, target, mask, idx):
    """The layer's loss in double precision with the experts as chosen, and its gradients."""
    p = {n: v.double().requires_grad_() for n, v in layer.params.items()}
    table = torch.where((torch.arange(layer.V, device=ids.device) == 0)[:, None], p["table"].detach(), p["table"])
    x = table[ids] * layer.scale
    s = torch.sigmoid(x @ p["router"].t()).gather(1, idx.long())
    w = 2.0 * s / s.sum(1, keepdim=True)
    out = 0
    for j in range(layer.k):
        e = idx[:, j].long()
        z = torch.einsum("th,tfh->tf", x, p["gate_up"][e])
        h = torch.nn.functional.silu(z[:, : layer.F]) * z[:, layer.F:]
        out = out + w[:, j, None] * (torch.einsum("tf,thf->th", h, p["down"][e]) + p["down_bias"][e])
    lz = out @ p["head"]
    m = mask.double()
    loss = ((torch.logsumexp(lz, 1) - lz.gather(1, target[:, None])[:, 0]) * m).sum() / m.sum()
    loss.backward()
    return float(loss.detach()), {n: v.grad for n, v in p.items()}


def test_layer_gradients_match_double_precision_autograd():
    """BF16 roundings (x, h, y, out, dout, dy, dzz, dxd, dx: nine on the longest path) are relative 2^-8 at most of the
    value each rounds, so a gradient differs by at most about 9 x 2^-8 of its norm."""
    import train_moe_experts as ex
    layer = ex.Layer(max_tokens=512, seed=3)
    layer.bias.normal_(0.0, 0.05, generator=torch.Generator(device="cuda").manual_seed(2))
    g = torch.Generator(device="cuda").manual_seed(5)
    follow = torch.arange(layer.V, device="cuda").roll(-1)
    follow[0], follow[-1] = 0, 1
    ids, target, mask = ex.batch(follow, 8, 64, g)
    s = layer.pool.stream
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        loss = layer.step(ids, target, mask)
        x = ap.embed(layer.params["table"], ids, scale=layer.scale)
        idx, _ = ap.route_scored(x.float() @ layer.params["router"].float().t(), layer.k, bias=layer.bias, groups=layer.groups,
                                 top_groups=layer.top_groups)
    torch.cuda.synchronize()
    e, grads = reference(layer, ids, target, mask, idx)
    assert int(layer.status) == 0
    assert abs(float(loss) - e) <= 9 * 2.0 ** -8 * e
    assert int(layer.counts.sum()) == int(mask.sum()) * layer.k
    for n, ge in grads.items():
        err = float((layer.grads[n].double() - ge).norm() / ge.norm())
        assert err <= 9 * 2.0 ** -8, (n, err)
    # one update: every master copy follows the step's formula from these gradients
    before = [m.double() for m in layer.opt.master]
    norm = float(torch.sqrt(sum((v.double() ** 2).sum() for v in layer.grads.values())))
    kept = [v.double() for v in layer.grads.values()]
    with torch.cuda.stream(s):
        layer.update()
    torch.cuda.synchronize()
    clip = min(1.0, 1.0 / norm)
    for m, b, v in zip(layer.opt.master, before, kept):
        v = v * clip
        new = b * (1 - 2e-2 * 0.01) - 2e-2 * v / (v.abs() + 1e-8)  # the first step: m / (1 - b1) = v, likewise its square
        # single precision: 64 roundings of 2^-24 of either term; gradients near eps turn on their last bits
        assert bool(((m.double() - new).abs() <= 64 * 2.0 ** -24 * (b.abs() + 2e-2)).all())
    assert not layer.counts.any() and all(not v.any() for v in layer.grads.values())


def test_example_runs():
    import train_moe_experts as ex
    h = ex.train(steps=12)
    assert all(loss == loss and loss < 20.0 for loss, _ in h)
    assert all(sum(c) > 0 for _, c in h)


def test_overflowing_pool_skips_the_update():
    import train_moe_experts as ex
    layer = ex.Layer(max_tokens=16, seed=1)  # room for 16 tokens' rows
    g = torch.Generator(device="cuda").manual_seed(5)
    follow = torch.arange(layer.V, device="cuda").roll(-1)
    ids, target, mask = ex.batch(follow, 8, 64, g)
    s = layer.pool.stream
    s.wait_stream(torch.cuda.current_stream())
    kept = [p.clone() for p in layer.params.values()]
    with torch.cuda.stream(s):
        layer.step(ids, target, mask)
        layer.update()
    torch.cuda.synchronize()
    assert layer.pool.overflow() != 0
    assert int(layer.opt.state["step"][0]) == 0
    assert all(torch.equal(a, b) for a, b in zip(kept, layer.params.values()))


def test_captured_step():
    """Forward, backward and update of the layer's own operators in one graph, replayed with other tokens."""
    T, E, k, H, F = 200, 8, 2, 64, 48
    g = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda *n, s=1.0: torch.randn(*n, generator=g, device="cuda") * s  # noqa: E731
    x, logits, dout = rnd(T, H).bfloat16(), rnd(T, E), rnd(T, H, s=0.1).bfloat16()
    W = rnd(E, H, H, s=H ** -0.5).bfloat16()
    bias, counts = torch.zeros(E, device="cuda"), torch.zeros(E, dtype=torch.int32, device="cuda")
    dW = torch.zeros(E, H, H, device="cuda")
    opt = ap.AdamW([W], [dW], lr=1e-2, master=True, state_bits=8)
    d = ap.dispatch_permute(x, ap.route_scored(logits, k)[0], E)
    out = {n: t for n, t in d.items()}
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    y, dy = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
    res, dl = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, E, device="cuda")
    dw = torch.zeros(T, k, device="cuda")

    def step():
        ap.route_scored(logits, k, bias=bias, groups=2, top_groups=1, counts=counts, idx=idx, w=w)
        ap.dispatch_permute(x, idx, E, out=out)
        ap.expert_linear(out["xd"], W, out["seg_off"], out["live"], act="silu", out=y)
        ap.combine_unpermute(y, out["dest"], w, out=res)
        ap.combine_backward(dout, y, out["dest"], w, dy=dy, dw=dw)
        ap.expert_linear_dw(dy, out["xd"], out["seg_off"], out["live"], dW=dW)
        ap.route_scored_backward(logits, idx, dw, dlogits=dl)
        opt.step(scale=opt.grad_norm(0.5)[1:])
        ap.route_bias_step(bias, counts, 1e-2, reset=True)
    state = [W, opt.master[0], bias] + [opt.state[n] for n in sorted(opt.state)]
    step()  # (allocates what the calls keep)
    torch.cuda.synchronize()
    first = [t.clone() for t in state]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    tokens = [(rnd(T, H).bfloat16(), rnd(T, E)) for _ in range(3)]
    results = []
    for run in (graph.replay, step):
        for t, v in zip(state, first):
            t.copy_(v)
        counts.zero_()
        for a, b in tokens:
            x.copy_(a), logits.copy_(b)
            run()
        torch.cuda.synchronize()
        results.append([t.clone() for t in state] + [res.clone(), dl.clone()])
    assert all(torch.equal(a, b) for a, b in zip(*results))
