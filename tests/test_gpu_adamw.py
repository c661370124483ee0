"""GPU parity: the AdamW step, its 8-bit moments, and the gradients' norm, against
their 64-bit plain forms.

Bounds (u = 2^-24, a rounding of single precision): m = b1 m + (1 - b1) g' takes
the constants' roundings, the scaling of g, a product and the sum: 5 u of the
magnitudes |b1 m| + |(1 - b1) g'|, called dm; v likewise 6 u of itself (its terms
do not cancel).  p takes 4 u of |p| (decay factor, product, sum) and of the change
32 u (two corrections by expm1 of 4 u each, root 4 u and 3 u of v, quotient 4 u,
products) and rate / denominator times dm.  BF16 results round by 2^-8 more.
Codes: x = |m| / m_scale has dm / m_scale and 8 u (block maximum, constant,
reciprocal, product), its root 4 u, and the sum with the fraction rounds at 256:
the code is the floor of a value in that range.
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
HYPER = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-6, weight_decay=0.1)
SIZES = [1, 7, 0, 255, 256, 257, 5000, 3, 2048, 66001]


def f64(t):
    return t.detach().double().cpu().numpy().ravel()


def make(sizes, kind, gkind, master, bits, offset=0, seed=1, **more):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def tensors(scale, dtype):
        got = []
        for n in sizes:  # `offset`: elements before each, so that it begins between vectors
            t = (torch.randn(n + offset, generator=g, device="cuda") * scale).to(dtype)
            got.append(t[offset:])
        return got
    params = tensors(0.5, kind)
    return ap.AdamW(params, tensors(1e-2, gkind), master=True if master else None, state_bits=bits, seed=77, **(HYPER | more))


def snapshot(o):
    s = {n: t.clone() for n, t in o.state.items()}
    return [f64(p) for p in (o.master or o.params)], {n: host(t) for n, t in s.items()}


def check_step(o, lr=None, scale=1.0, **call):
    before, old = snapshot(o)
    o.step(lr=lr, **call)
    torch.cuda.synchronize()
    lr = HYPER["lr"] if lr is None else float(lr)
    t = int(old["step"][0]) + 1
    assert host(o.state["step"]).tolist() == [t, 0]
    new = {n: host(x) for n, x in o.state.items()}
    b1, b2 = HYPER["betas"]
    for i, ((at, n), p0, g) in enumerate(zip(o.parts, before, o.grads)):
        if not n:
            continue
        blk = slice(at // 256, -(-(at + n) // 256))
        if o.state_bits == 8:
            m0, v0 = layer.adamw_decode(old["m"][at:at + n], old["v"][at:at + n], old["m_scale"][blk], old["v_scale"][blk])
        else:
            m0, v0 = old["m"][at:at + n].astype(np.float64), old["v"][at:at + n].astype(np.float64)
        gf = f64(g)
        p, m, v, change = layer.adamw_step(p0, gf, m0, v0, t, lr, HYPER["betas"], HYPER["eps"], HYPER["weight_decay"], scale)
        dm = 5 * U * (np.abs(b1 * m0) + np.abs((1 - b1) * gf * scale)) + 2.0 ** -140
        rate = lr / (1 - b1 ** t) / (np.sqrt(v / (1 - b2 ** t)) + HYPER["eps"])
        bound = 4 * U * np.abs(p0) + 32 * U * np.abs(change) + rate * dm
        if o.master is not None:
            assert np.all(np.abs(f64(o.master[i]) - p) <= bound)
            assert torch.equal(o.params[i], o.master[i].bfloat16())
        else:
            half = 2.0 ** -8 * np.abs(p) if o.params[i].dtype == torch.bfloat16 else 0.0
            assert np.all(np.abs(f64(o.params[i]) - p) <= bound * 1.01 + half)
        if o.state_bits == 32:
            assert np.all(np.abs(new["m"][at:at + n] - m) <= dm)
            assert np.all(np.abs(new["v"][at:at + n] - v) <= 6 * U * v + 2.0 ** -140)
            continue
        low, high = layer.adamw_noise(77, t, i, n)
        for name, x, dx, top, r in (("m", np.abs(m), dm, 127, low), ("v", np.sqrt(v), 8 * U * np.sqrt(v), 255, high)):
            s = layer.block_max(x) / top ** 2
            ds = layer.block_max(dx) / top ** 2 + 4 * U * s
            assert np.all(np.abs(new[name + "_scale"][blk] - s) <= ds)
            each, deach = np.repeat(s, 256)[:n], np.repeat(ds, 256)[:n]
            code = np.abs(new[name][at:at + n].astype(np.int64))
            with np.errstate(divide="ignore", invalid="ignore"):
                lo = np.where(each > 0, np.maximum(x - dx, 0) / (each + deach) * (1 - 8 * U), 0.0)
                hi = np.where(each > 0, (x + dx) / (each - deach) * (1 + 8 * U), 0.0)
            lo = np.floor(np.sqrt(lo) * (1 - 4 * U) + r - 256 * U)
            hi = np.floor(np.sqrt(hi) * (1 + 4 * U) + r + 256 * U)
            if name == "v":
                lo, hi = np.where(x > 0, np.maximum(lo, 1), lo), np.where(x > 0, np.maximum(hi, 1), hi)
            on = each > 0
            assert np.all(((code >= np.minimum(lo, top)) & (code <= np.minimum(hi, top)))[on])
            assert not code[~on].any()
        sign = np.sign(new["m"][at:at + n].astype(np.float64))
        assert np.all((sign == np.sign(m)) | (sign == 0) | (np.abs(m) <= dm))


@pytest.mark.parametrize("kind,gkind,master", [(torch.float32, torch.float32, False), (torch.float32, torch.bfloat16, False),
                                               (torch.bfloat16, torch.bfloat16, False), (torch.bfloat16, torch.float32, True),
                                               (torch.bfloat16, torch.bfloat16, True), (torch.bfloat16, torch.float32, False)])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("offset", [0, 1])
def test_steps(kind, gkind, master, bits, offset):
    o = make(SIZES, kind, gkind, master, bits, offset)
    for step in range(4):
        if step == 2:
            for g in o.grads:
                g.mul_(-3.0)
        check_step(o)


@pytest.mark.parametrize("count", [57, 441, 1000])
@pytest.mark.parametrize("bits", [8, 32])
def test_many_tensors(count, bits):
    """More tensors than one launch's table takes: 56 and 440."""
    sizes = [(i * 37) % 600 for i in range(count)]
    o = make(sizes, torch.float32, torch.float32, False, bits)
    n0 = ap.launch_count()
    check_step(o)
    assert ap.launch_count() - n0 == -(-count // 440)
    check_step(o)


@pytest.mark.parametrize("bits", [8, 32])
def test_long_run_of_steps(bits):
    """Step numbers whose corrections are near 0 and near 1."""
    o = make([300], torch.float32, torch.float32, False, bits)
    for t in (0, 1, 9, 999, 10 ** 6, 2 ** 24 + 1, 2 ** 30):
        o.state["step"].copy_(torch.tensor([t, 0], dtype=torch.int32))
        check_step(o)


def test_arguments_on_the_gpu():
    o = make(SIZES, torch.float32, torch.float32, False, 32)
    check_step(o, lr=torch.tensor(3e-3, device="cuda"))
    word = torch.tensor([0.25], device="cuda")
    before, old = snapshot(o)
    o.step(scale=word)
    torch.cuda.synchronize()
    (at, n), g = o.parts[6], f64(o.grads[6])
    p, _, _, _ = layer.adamw_step(before[6], g, old["m"][at:at + n].astype(np.float64), old["v"][at:at + n].astype(np.float64), 2,
                                  HYPER["lr"], HYPER["betas"], HYPER["eps"], HYPER["weight_decay"], 0.25)
    assert np.all(np.abs(f64(o.params[6]) - p) <= 64 * U * (np.abs(p) + HYPER["lr"]))


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("why", ["word", "scale", "pool"])
def test_skipped_steps_change_nothing(bits, why):
    o = make(SIZES, torch.bfloat16, torch.float32, True, bits)
    check_step(o)
    kept = [t.clone() for t in o.params + o.master] + [t.clone() for t in o.state.values()]
    if why == "word":
        o.step(skip=torch.tensor([4], dtype=torch.int32, device="cuda"))
    elif why == "scale":
        for bad in (float("nan"), float("inf"), -float("inf")):
            o.step(scale=torch.tensor([bad], device="cuda"))
    else:
        pool = ap.Pool(4, 4 * 64, 1, 1, 2, 1)
        x = torch.zeros(8, 32, dtype=torch.bfloat16, device="cuda")  # 64-byte rows, two pages' worth into one page
        seg, live = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), 8, dtype=torch.int32, device="cuda")
        pool.stream.wait_stream(torch.cuda.current_stream())
        pool.push(0, [x], seg, live)
        torch.cuda.synchronize()
        o.step(skip=pool)
    torch.cuda.synchronize()
    for a, b in zip(kept, o.params + o.master + list(o.state.values())):
        assert torch.equal(a, b)
    if why == "word":
        o.step(skip=torch.tensor([0], dtype=torch.int32, device="cuda"))
        assert int(o.state["step"][0]) == 2


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,offset", [([1], 0), (SIZES, 0), (SIZES, 1), ([0, 0], 0), ([4_000_001], 0), ([100] * 500, 0)])
def test_norm(kind, sizes, offset):
    """Each square and the fused sums of eight round by 8 u of the sum, the rest is as exact as double."""
    o = make(sizes, torch.float32, kind, False, 32, offset)
    e = float(np.sqrt(sum((f64(g) ** 2).sum() for g in o.grads)))
    got = host(o.grad_norm())
    assert abs(got[0] - e) <= 6 * U * e and got[1] == 1.0
    if e:
        got = host(o.grad_norm(e / 3))
        assert abs(got[1] - 1 / 3) <= 8 * U
        assert host(o.grad_norm(e * 3))[1] == 1.0
    again = torch.empty(2, device="cuda")
    assert torch.equal(o.grad_norm(out=again), o.grad_norm())
    assert o.grad_norm() is o.grad_norm()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38])
def test_norm_that_is_not_finite_skips_the_step(bad):
    o = make(SIZES, torch.float32, torch.float32, False, 8)
    o.grads[6][1234] = bad
    out = o.grad_norm(1.0)
    assert np.isnan(host(out)[1])
    before, _ = snapshot(o)
    o.step(scale=out[1:])
    after, _ = snapshot(o)
    assert all(np.array_equal(a, b) for a, b in zip(before, after)) and not o.state["step"].any()


def test_moments_read_out():
    o = make(SIZES, torch.float32, torch.float32, False, 8)
    for _ in range(3):
        o.step()
    s = {n: host(t) for n, t in o.state.items()}
    m, v = layer.adamw_decode(s["m"], s["v"], s["m_scale"], s["v_scale"])
    for dtype, half in ((torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)):
        gm, gv = o.moments(dtype)
        assert gm.dtype == dtype
        # the product with the scale rounds once, the square of the root twice more
        assert np.all(np.abs(f64(gm) - m) <= (2 * U + half) * np.abs(m) * 1.01 + 2.0 ** -140)
        assert np.all(np.abs(f64(gv) - v) <= (4 * U + half) * v * 1.01 + 2.0 ** -140)
    o32 = make(SIZES, torch.float32, torch.float32, False, 32)
    assert o32.moments()[0] is o32.state["m"]


def test_codes_behind_a_tensor_do_not_matter():
    def run(fill):
        o = make([300, 5], torch.float32, torch.float32, False, 8)
        o.step()
        for at, n in o.parts:
            end = -(-(at + n) // 256) * 256
            for name in ("m", "v"):
                o.state[name][at + n:end] = fill
        o.step()
        return o
    a, b = run(0), run(100)
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))
    assert torch.equal(a.state["m_scale"], b.state["m_scale"]) and torch.equal(a.state["v_scale"], b.state["v_scale"])


def test_blocks_of_zeros_and_of_nan():
    o = make([600], torch.float32, torch.float32, False, 8)
    o.grads[0].zero_()
    o.step()
    assert not o.state["m"].any() and not o.state["v"].any() and not o.state["v_scale"].any()
    o.grads[0].fill_(1e-3)
    o.grads[0][300] = float("nan")
    o.step()
    m, v = o.moments()
    nan = torch.isnan(m)
    assert nan[256:512].all() and not nan[:256].any() and not nan[512:].any() and torch.equal(nan, torch.isnan(v))


def test_coded_moments_follow_the_gradients():
    """Codes rounded at random keep the mean: after many steps of one gradient's size, sqrt(v) is near it although each
    step moves v by less than a code.  A step's rounding is at most a code: of c near 200 in sqrt(v) = s c^2 it moves v by
    4 / 200; steps decay with 0.999, so the error's deviation is below 4 / 200 / 2 / sqrt(2 * 0.001) = 22%, and the mean
    over 4096 elements lies within 22% / 64 * 5 < 2%."""
    n = 4096
    o = ap.AdamW([torch.zeros(n, device="cuda")], [torch.full((n,), 1e-3, device="cuda")], betas=(0.9, 0.999), state_bits=8)
    o.grads[0][::256] = 1.5e-3  # the block's largest, so that the others' codes lie between
    for _ in range(1500):
        o.step()
    v = o.moments()[1].view(-1, 256)[:, 1:].double()
    expected = 1e-6 * (1 - 0.999 ** 1500)
    assert abs(float(v.mean()) / expected - 1) <= 0.02
    o.grads[0].mul_(0.1)
    for _ in range(1500):
        o.step()
    v = o.moments()[1].view(-1, 256)[:, 1:].double()
    expected = expected * 0.999 ** 1500 + 1e-8 * (1 - 0.999 ** 1500)
    assert abs(float(v.mean()) / expected - 1) <= 0.05


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_and_replayed(bits):
    a, b = (make(SIZES, torch.bfloat16, torch.bfloat16, True, bits) for _ in range(2))
    lr, out = torch.tensor(1e-2, device="cuda"), torch.empty(2, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.grad_norm(0.5, out=out)
        a.step(lr=lr, scale=out[1:])
    for step in range(4):
        lr.fill_(1e-2 / (step + 1))
        for x, y in zip(a.grads, b.grads):
            x.mul_(0.7)
            y.mul_(0.7)
        g.replay()
        b.step(lr=lr, scale=b.grad_norm(0.5)[1:])
    torch.cuda.synchronize()
    for x, y in zip(a.params + a.master + list(a.state.values()), b.params + b.master + list(b.state.values())):
        assert torch.equal(x, y)
    assert int(a.state["step"][0]) == 4


def test_another_stream():
    o = make(SIZES, torch.float32, torch.float32, False, 32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o.step(scale=o.grad_norm(1.0, stream=s)[1:], stream=s)
    torch.cuda.synchronize()
    assert int(o.state["step"][0]) == 1


def test_checkpoint_continues():
    a = make(SIZES, torch.float32, torch.float32, False, 8)
    a.step()
    b = ap.AdamW([p.clone() for p in a.params], [g.clone() for g in a.grads], state_bits=8, seed=77,
                 state={n: t.clone() for n, t in a.state.items()}, **HYPER)
    a.step()
    b.step()
    for x, y in zip(a.params + list(a.state.values()), b.params + list(b.state.values())):
        assert torch.equal(x, y)


def test_refusals():
    p, g = torch.zeros(10, device="cuda"), torch.zeros(10, device="cuda")
    for match, call in (
            ("empty", lambda: ap.AdamW([], [])),
            ("state_bits", lambda: ap.AdamW([p], [g], state_bits=16)),
            ("float", lambda: ap.AdamW([p.half()], [g])),
            ("contiguous", lambda: ap.AdamW([torch.zeros(5, 4, device="cuda").t()], [torch.zeros(4, 5, device="cuda")])),
            ("share", lambda: ap.AdamW([p, p[2:5]], [g, g[2:5]])),
            ("grads", lambda: ap.AdamW([p], [])),
            ("grads", lambda: ap.AdamW([p], [g[:9]])),
            ("grads", lambda: ap.AdamW([p], [g.half()])),
            ("CUDA", lambda: ap.AdamW([p.cpu()], [g])),
            ("master", lambda: ap.AdamW([p], [g], master=True)),
            ("master", lambda: ap.AdamW([p.bfloat16()], [g], master=[])),
            ("state m", lambda: ap.AdamW([p], [g], state={"m": torch.zeros(10, device="cuda")})),
            ("one float32", lambda: ap.AdamW([p], [g]).step(scale=torch.zeros(2, device="cuda"))),
            ("one float32", lambda: ap.AdamW([p], [g]).step(lr=torch.zeros(1))),
            ("status", lambda: ap.AdamW([p], [g]).step(skip=torch.zeros(1, dtype=torch.int32))),
            ("max_norm", lambda: ap.AdamW([p], [g]).grad_norm(0.0)),
            ("moments", lambda: ap.AdamW([p], [g]).moments(torch.bfloat16))):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(ap.APError, match="beta"):
        ap.AdamW([p], [g], betas=(1.0, 0.9)).step()
