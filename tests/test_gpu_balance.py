"""GPU parity: routing with its balance loss, and the router's gradient, against
their 64-bit plain forms.

Ids and counts are compared exactly.  The bounds of the other outputs follow
from the kernels' single-precision steps (u = 2^-24, d the largest distance of
a logit from its row's maximum that matters):

* p: the difference l - m rounds once (relative u of |l - m| in the exponent),
  exp is within 2 ulp (counted as 4 u), the row's sum has E/32 + 5 additions of
  terms with that error, then a reciprocal and a product: relative
  (2 d + 8 + E/32 + 5 + 4) u, below P_REL;
* prob: a warp adds at most S/8 + 1 rows, then 8 warps, at most 608/8 + 1
  blocks and 8 parts, and one division: P_REL + (S/8 + 100) u;
* slope: ten roundings; loss: sums of prob * slope over E and the groups.
"""
import numpy as np
import pytest
import torch

import oracle
from activation_paging_gb300 import inputs
from gpu_util import host, route_tolerance, to_dev
from oracle import training

pytestmark = pytest.mark.gpu

ap = pytest.importorskip("activation_paging_gb300")

U = 2.0 ** -24


def p_rel(logits):
    """Per row: relative error of a softmax value (values below e^-87 may flush to zero: absolute 2^-125)."""
    x = logits.astype(np.float64)
    fine = np.isfinite(x)
    d = np.maximum(np.where(fine, x, -np.inf).max(1) - np.where(fine, x, np.inf).min(1), 0.0)
    return ((2 * np.minimum(d, 90.0) + 17 + logits.shape[1] / 32) * U)[:, None]


def check_balance(logits, k, coef, S, mask, out=None, stream=None):
    T, E = logits.shape
    m = None if mask is None else to_dev(mask)
    r = ap.route_balance(to_dev(logits), k, coef=coef, group_tokens=S, mask=m, out=out, stream=stream)
    torch.cuda.synchronize()
    seen = logits if mask is None else np.where(mask[:, None].astype(bool), logits, 0).astype(np.float32)
    e = training.route_balance(seen, k, coef, S, mask)
    S1, G = training._groups(T, S)
    on = training.counting(logits, mask)
    live = on if mask is not None else np.ones(T, bool)
    assert np.array_equal(host(r["idx"])[live], e["idx"][live])
    wt = route_tolerance(np.where(np.isfinite(seen), seen, np.float32(-1e4)), e["idx"], e["w"])
    assert np.all(np.abs(host(r["w"])[live] - e["w"][live]) <= wt[live] + 2.0 ** -24 * e["w"][live])
    assert np.array_equal(host(r["counts"]), e["counts"])
    rel = float(p_rel(seen).max()) if T else 0.0
    prel = rel + (S1 / 8 + 100) * U
    assert np.all(np.abs(host(r["prob"]) - e["prob"]) <= prel * e["prob"] + 2.0 ** -120)
    assert np.all(np.abs(host(r["slope"]) - e["slope"]) <= 10 * U * np.abs(e["slope"]))
    terms = abs(coef)
    bound = (prel + (10 + 13 + G * E / 32 / 256 + 8) * U) * max(abs(e["loss"]), terms * 1e-3)
    assert abs(float(r["loss"]) - e["loss"]) <= bound
    return r, e


@pytest.mark.parametrize("T,E,k,S,pad", [
    (1, 1, 1, 0, False),
    (1, 8, 8, 0, False),
    (7, 5, 3, 3, False),          # odd everything, a short last group
    (256, 8, 2, 0, False),
    (999, 60, 6, 333, True),
    (1000, 128, 8, 1, True),      # a group per token
    (4097, 33, 4, 1024, True),
    (2048, 256, 8, 512, True),
    (300, 511, 32, 100, False),
    (130, 1024, 12, 64, True),
    (20000, 64, 6, 0, True),
])
def test_route_balance_matches_plain_form(T, E, k, S, pad):
    logits = inputs.router_logits(T + E, T, E, 1.0, 0.4)
    mask = None
    if pad:
        S1, G = training._groups(T, S)
        length = inputs.rng(T, 7).integers(0, S1 + 1, G)
        if G > 2:
            length[1] = 0  # a group whose mask leaves nothing
        mask = ((np.arange(T) % S1) < length[np.arange(T) // S1]).astype(np.uint8)
    check_balance(logits, k, 0.01, S, mask)


def test_route_balance_routes_as_route_topk():
    logits = inputs.router_logits(4, 5000, 128)
    logits[:, 17] = logits[:, 90]
    logits[100:200] = np.round(logits[100:200])  # many ties
    idx, w = ap.route_topk(to_dev(logits), 8)
    mask = torch.arange(5000, device="cuda") % 3 != 0
    r = ap.route_balance(to_dev(logits), 8, mask=mask)
    assert torch.equal(r["idx"], idx) and torch.equal(r["w"], w)


def test_route_balance_no_tokens_and_no_counting_tokens():
    r = ap.route_balance(torch.empty(0, 16, device="cuda"), 2)
    assert float(r["loss"]) == 0 and r["counts"].shape == (0, 16)
    logits = inputs.router_logits(1, 40, 16)
    r = ap.route_balance(to_dev(logits), 2, group_tokens=7, mask=torch.zeros(40, dtype=torch.bool, device="cuda"))
    assert float(r["loss"]) == 0
    for n in ("counts", "prob", "slope"):
        assert not host(r[n]).any()
    assert np.array_equal(host(r["idx"]), oracle.route_topk(logits, 2)[0])


def test_route_balance_masked_experts_and_rows():
    """-infinity and the type's lowest value on experts; whole rows of either; NaN where the mask hides it."""
    T, E, k = 200, 40, 4
    logits = inputs.router_logits(8, T, E)
    logits[:, 5] = -np.inf
    logits[3, 2:] = -np.inf                       # fewer than k experts left
    logits[10] = -np.inf                          # none left: the row does not count
    logits[11] = np.finfo(np.float32).min         # all equal: uniform
    logits[12, ::2] = np.finfo(np.float32).min
    mask = np.ones(T, np.uint8)
    mask[20:25] = 0
    logits[20] = np.nan
    logits[21, 3] = np.inf
    r, e = check_balance(logits, k, 0.5, 50, mask)
    w, idx = host(r["w"]), host(r["idx"])
    assert np.all(w[10] == 0)
    assert np.all(w[3, 2:] == 0) and abs(w[3].sum() - 1) < 1e-6
    assert np.all((idx >= 0) & (idx < E))
    assert np.all(host(r["prob"])[1:, 5] == 0)  # (row 11 gives expert 5 its share in the first group)


def test_equal_inputs_give_equal_bits():
    logits = to_dev(inputs.router_logits(2, 30000, 128, 1.0, 0.4))
    a = ap.route_balance(logits, 8, coef=0.01, group_tokens=4096)
    for _ in range(5):
        b = ap.route_balance(logits, 8, coef=0.01, group_tokens=4096)
        for n in ("prob", "slope", "loss", "counts"):
            assert torch.equal(a[n], b[n])


def grad_bound(logits, idx, w, dw, slope, dloss, S, mask):
    """|error| of dlogits: q = g p (s - <p, s>) with p's relative error twice (numerator of q, and through the mean),
    E/32 + 5 additions in <p, s>, five products; z = w (dw - <w, dw>) with five additions and two products."""
    T, E = logits.shape
    rel = p_rel(logits)
    b = np.zeros((T, E))
    if slope is not None:
        p = training.softmax(logits)
        s = np.abs(slope.astype(np.float64)[np.arange(T) // S])
        mean = (p * s).sum(1, keepdims=True)
        b += abs(dloss) * p * (s + mean) * (3 * rel + (E / 32 + 12) * U)
    if dw is not None:
        z = np.abs(w) * (np.abs(dw) + np.abs(w * dw).sum(1, keepdims=True)) * 10 * U
        full = np.abs(w) * (np.abs(dw) + np.abs(w * dw).sum(1, keepdims=True)) * U
        np.add.at(b, (np.arange(T)[:, None], idx), z + full)
    return b * (1 + 1e-6) + 2.0 ** -120


@pytest.mark.parametrize("T,E,k,S,pad,terms", [
    (1, 1, 1, 0, False, "both"),
    (1, 8, 8, 0, False, "both"),
    (7, 5, 3, 3, False, "both"),
    (256, 8, 2, 0, False, "both"),
    (999, 60, 6, 333, True, "both"),
    (1000, 128, 8, 1, True, "both"),
    (513, 130, 4, 100, True, "both"),     # E % 4 != 0: scalar loads
    (2048, 256, 8, 512, True, "both"),
    (300, 511, 32, 100, False, "both"),
    (130, 1024, 12, 64, True, "both"),
    (70, 1023, 3, 0, True, "both"),
    (500, 64, 6, 0, True, "dw"),
    (500, 64, 6, 50, True, "slope"),
    (50, 64, 6, 0, False, "none"),
])
def test_route_backward_matches_plain_form(T, E, k, S, pad, terms):
    logits = inputs.router_logits(T + 3 * E, T, E, 1.0, 0.4)
    S1, G = training._groups(T, S)
    mask = (inputs.rng(T, 7).random(T) < 0.8).astype(np.uint8) if pad else None
    e = training.route_balance(logits, k, 0.3, S, mask)
    w, slope = e["w"].astype(np.float32), e["slope"].astype(np.float32)
    dw = inputs.rng(T, 11).standard_normal((T, k)).astype(np.float32) * np.float32(0.1)
    dloss = np.float32(-1.75)
    if terms in ("dw", "none"):
        slope = None
    if terms in ("slope", "none"):
        dw = None
    got = ap.route_backward(to_dev(logits), to_dev(e["idx"]), to_dev(w), None if dw is None else to_dev(dw),
                            None if slope is None else to_dev(slope), to_dev(np.array([dloss])), S,
                            None if mask is None else to_dev(mask))
    exp = training.route_backward(logits, e["idx"], w, dw, slope, float(dloss), S, mask)
    bound = grad_bound(logits, e["idx"], w, dw, slope, float(dloss), S1, mask)
    assert np.all(np.abs(host(got) - exp) <= bound)


def test_route_backward_in_place_masks_and_bad_ids():
    T, E, k = 100, 24, 3
    logits = inputs.router_logits(6, T, E)
    logits[:, 4] = -np.inf
    logits[7] = -np.inf
    mask = np.ones(T, np.uint8)
    mask[9] = 0
    e = training.route_balance(logits, k, 1.0, 0, mask)
    w, slope, idx = e["w"].astype(np.float32), e["slope"].astype(np.float32), e["idx"].copy()
    dw = inputs.rng(3, 3).standard_normal((T, k)).astype(np.float32)
    idx[5, 1], idx[6, 0] = -1, E
    exp = training.route_backward(logits, idx, w, dw, slope, 1.0, 0, mask)
    hidden = logits.copy()
    hidden[9] = np.nan  # masked: its logits reach nothing
    buf = to_dev(hidden)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ap.route_backward(buf, to_dev(idx), to_dev(w), to_dev(dw), to_dev(slope), mask=to_dev(mask), dlogits=buf,
                            status=status)
    assert got.data_ptr() == buf.data_ptr()
    assert int(host(status)[0]) == ap.FLAG_BAD_INDEX
    ok = np.where((idx >= 0) & (idx < E), idx, 0)
    bound = grad_bound(np.where(np.isfinite(logits), logits, np.float32(-80)), ok, w, dw, slope, 1.0, T, mask)
    assert np.all(np.isfinite(host(got)))
    assert np.all(np.abs(host(got) - exp) <= bound)
    assert np.all(host(got)[7][np.setdiff1d(np.arange(E), idx[7])] == 0)


def test_route_backward_matches_differences_of_the_forward_kernel():
    """Central differences of <dw, w> + dloss * loss through route_balance, step 2^-6, counts held by keeping the
    chosen experts apart: error O(h^2) of third derivatives (below 1) plus rounding u / h of O(1) values."""
    T, E, k, h = 6, 8, 2, 2.0 ** -6
    logits = np.zeros((T, E), np.float32)
    for t in range(T):
        logits[t] = (np.roll(np.arange(E), 3 * t) * 0.5).astype(np.float32)
    dw = inputs.rng(5, 5).standard_normal((T, k)).astype(np.float32)
    r = ap.route_balance(to_dev(logits), k, coef=1.0)
    d = host(ap.route_backward(to_dev(logits), r["idx"], r["w"], to_dev(dw), r["slope"]))
    for t in range(T):
        for e in range(E):
            f = []
            for s in (h, -h):
                x = logits.copy()
                x[t, e] += np.float32(s)
                q = ap.route_balance(to_dev(x), k, coef=1.0)
                assert torch.equal(q["idx"], r["idx"])
                f.append(float((host(q["w"]).astype(np.float64) * dw).sum()) + float(q["loss"]))
            # |third derivative| of a softmax-weighted sum of values of magnitude at most M is below M
            most = np.abs(dw).sum() + float(r["slope"].abs().max()) * 4
            assert abs((f[0] - f[1]) / (2 * h) - d[t, e]) <= most * h * h / 6 + 64 * U / h * most


def test_route_balance_on_another_stream_and_in_a_graph():
    logits = to_dev(inputs.router_logits(2, 4096, 64))
    a = ap.route_balance(logits, 6, coef=0.1, group_tokens=512)
    da = ap.route_backward(logits, a["idx"], a["w"], a["w"], a["slope"], group_tokens=512)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = ap.route_balance(logits, 6, coef=0.1, group_tokens=512, stream=s)
    db = ap.route_backward(logits, b["idx"], b["w"], b["w"], b["slope"], group_tokens=512, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(da, db) and torch.equal(a["loss"], b["loss"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = ap.route_balance(logits, 6, coef=0.1, group_tokens=512)
        dc = ap.route_backward(logits, c["idx"], c["w"], c["w"], c["slope"], group_tokens=512)
    logits.copy_(to_dev(inputs.router_logits(77, 4096, 64)))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    a = ap.route_balance(logits, 6, coef=0.1, group_tokens=512)
    assert torch.equal(a["loss"], c["loss"]) and torch.equal(a["counts"], c["counts"])
    assert torch.equal(ap.route_backward(logits, a["idx"], a["w"], a["w"], a["slope"], group_tokens=512), dc)
