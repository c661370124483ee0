"""Offsets past 32 bits in routing by scores, the experts' products and the
weights' update: the far end of buffers of more than 2^31 elements, against the
same call on a copy of that end alone, whose results have the same bits.
"""
import pytest
import torch

import activation_paging_gb300 as ap

pytestmark = pytest.mark.gpu
BIG = 2 ** 31


@pytest.fixture(autouse=True)
def room():
    yield
    torch.cuda.empty_cache()


def gen(seed=1):
    return torch.Generator("cuda").manual_seed(seed)


def test_routing_of_many_tokens():
    E, k, tail = 256, 8, 1000
    T = BIG // E + tail
    logits = torch.zeros(T, E, device="cuda")
    logits[-tail:] = torch.randn(tail, E, generator=gen(), device="cuda")
    bias = torch.randn(E, generator=gen(2), device="cuda") * 0.01
    counts, few = (torch.zeros(E, dtype=torch.int32, device="cuda") for _ in range(2))
    args = dict(bias=bias, groups=8, top_groups=4, scale=2.5)
    idx, w = ap.route_scored(logits, k, counts=counts, **args)
    i, v = ap.route_scored(logits[-tail:].clone(), k, counts=few, **args)
    assert torch.equal(idx[-tail:], i) and torch.equal(w[-tail:], v)
    first = torch.bincount(idx[0].long(), minlength=E)
    assert torch.equal(counts.long(), few.long() + (T - tail) * first)
    dw = torch.zeros(T, k, device="cuda")
    dw[-tail:] = torch.randn(tail, k, generator=gen(3), device="cuda")
    want = ap.route_scored_backward(logits[-tail:].clone(), i, dw[-tail:].clone(), scale=2.5)
    got = ap.route_scored_backward(logits, idx, dw, scale=2.5, dlogits=logits)
    assert torch.equal(got[-tail:], want) and not got[:-tail].any()


@pytest.mark.parametrize("K", [64, 71])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_rows_of_the_products(K, act):
    """Few live rows at both ends of buffers whose results have more than 2^31 elements."""
    N, live = 1024, 300
    wide = 2 * N if act == "swiglu" else N
    rows = BIG // N + live
    W = torch.randn(2, wide, K, generator=gen(), device="cuda").bfloat16()
    bias = torch.randn(2, wide, generator=gen(2), device="cuda")
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    res = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    x[-live:] = torch.randn(live, K, generator=gen(3), device="cuda")
    res[-live:] = torch.randn(live, N, generator=gen(4), device="cuda")
    seg, n = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, rows - live], [17, live]))
    # the copy: the same average of rows for each expert, so the same tiles
    xs, rs = (torch.cat([t[:live], t[-live:]]) for t in (x, res))
    near = torch.tensor([0, live], dtype=torch.int32, device="cuda")

    pre = torch.zeros(rows, wide, dtype=torch.bfloat16, device="cuda")
    pres = torch.zeros(2 * live, wide, dtype=torch.bfloat16, device="cuda")
    y = ap.expert_linear(x, W, seg, n, bias=bias, act=act, residual=res, pre=pre)
    ys = ap.expert_linear(xs, W, near, n, bias=bias, act=act, residual=rs, pre=pres)
    assert torch.equal(y[-live:], ys[live:]) and torch.equal(pre[-live:], pres[live:])
    assert torch.equal(y[:17], ys[:17]) and torch.equal(pre[:17], pres[:17])
    del res, x, y

    # backwards through a product of K outputs and the activation
    dy = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    dy[-live:] = torch.randn(live, K, generator=gen(5), device="cuda")
    V = torch.randn(2, K, N, generator=gen(6), device="cuda").bfloat16()
    dx = ap.expert_linear_dx(dy, V, seg, n, act=act, pre=pre, out=pre)
    dxs = ap.expert_linear_dx(torch.cat([dy[:live], dy[-live:]]), V, near, n, act=act, pre=pres)
    assert torch.equal(dx[-live:], dxs[live:]) and torch.equal(dx[:17], dxs[:17])

    db, dbs = (torch.empty(2, wide, device="cuda") for _ in range(2))
    dW = ap.expert_linear_dw(dx, dy, seg, n, dbias=db)
    dWs = ap.expert_linear_dw(dxs, torch.cat([dy[:live], dy[-live:]]), near, n, dbias=dbs)
    assert torch.equal(dW, dWs) and torch.equal(db, dbs)


@pytest.mark.parametrize("K", [1048, 1041])
def test_weights_of_the_products(K):
    """The last of 1024 experts' weights, against the last of 8: as few rows for each, so the same tiles."""
    E, few, N, live = 1024, 8, 2048, 30
    W = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    W[-1] = torch.randn(N, K, generator=gen(), device="cuda")
    x = torch.randn(live, K, generator=gen(2), device="cuda").bfloat16()
    dy = torch.randn(live, N, generator=gen(3), device="cuda").bfloat16()
    seg = torch.zeros(E, dtype=torch.int32, device="cuda")
    n = seg.clone()
    n[-1] = live
    far, near = (seg, n), (seg[-few:].clone(), n[-few:].clone())
    V = W[-few:].clone()
    assert torch.equal(ap.expert_linear(x, W, *far), ap.expert_linear(x, V, *near))
    assert torch.equal(ap.expert_linear_dx(dy, W, *far), ap.expert_linear_dx(dy, V, *near))
    del W
    for dtype in (torch.float32, torch.bfloat16):
        dW = torch.zeros(E, N, K, dtype=dtype, device="cuda")
        ap.expert_linear_dw(dy, x, *far, dW=dW, accumulate=True)
        dV = torch.zeros(few, N, K, dtype=dtype, device="cuda")
        ap.expert_linear_dw(dy, x, *near, dW=dV, accumulate=True)
        assert torch.equal(dW[-few:], dV) and dV[-1].any()
        del dW


@pytest.mark.parametrize("kind,bits", [(torch.float32, 32), (torch.bfloat16, 8)])
def test_update_of_many_elements(kind, bits):
    tail = 1000
    p = torch.zeros(BIG + tail, dtype=kind, device="cuda")
    g = torch.zeros_like(p)
    p[BIG:] = torch.randn(tail, generator=gen(), device="cuda")
    g[BIG:] = torch.randn(tail, generator=gen(2), device="cuda")
    q, h = p[BIG:].clone(), g[BIG:].clone()
    far, near = ap.AdamW([p], [g], state_bits=bits), ap.AdamW([q], [h], state_bits=bits)
    norm = far.grad_norm(1.0)
    want = torch.linalg.vector_norm(h.double())
    assert abs(norm[0].item() - want.item()) <= 1e-6 * want.item()
    far.step(scale=norm[1:])
    near.step(scale=norm[1:])
    assert torch.equal(p[BIG:], q) and not p[:BIG].any()
    for name in ("m_scale", "v_scale") if bits == 8 else ("m", "v"):
        a, b = far.state[name], near.state[name]
        assert torch.equal(a[-b.numel():], b) and not a[:-b.numel()].any()
    if bits == 8:
        m, v = far.moments(torch.bfloat16)
        assert not m[:BIG].any() and not v[:BIG].any() and m[BIG:BIG + tail].any() and v[BIG:BIG + tail].any()
