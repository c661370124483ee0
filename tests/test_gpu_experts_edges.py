"""GPU: the experts' products at the edges of what a call may ask for.

Operands of small whole numbers: products and sums below 2^24 are exact in single precision, whatever their order, so
results are the exact ones (rounded once to BF16: by 2^-8 of themselves at most).  u = 2^-24."""
import numpy as np
import pytest
import torch

from gpu_util import host, to_dev
from oracle import layer

pytestmark = pytest.mark.gpu

ap = pytest.importorskip("activation_paging_gb300")

U = 2.0 ** -24
HALF = 2.0 ** -8


def whole(shape, low, high, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(low, high + 1, shape, generator=g, device="cuda", dtype=torch.int8).bfloat16()


def one(rows):
    return torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), rows, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weights_gradient_of_millions_of_rows(dtype):
    """One expert of 4 million rows: 65536 stages, in one section for BF16 results."""
    rows = (1 << 22) - 5
    dy, x, status = whole((rows, 64), 0, 1, 1), whole((rows, 64), -1, 1, 2), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ap.expert_linear_dw(dy, x, *one(rows), dtype=dtype, status=status)[0].double()
    want = sum(a.double().t() @ b.double() for a, b in zip(dy.split(1 << 18), x.split(1 << 18)))
    assert int(status) == 0
    assert float(want.abs().max()) < 2 ** 24
    assert bool(((got - want).abs() <= (HALF * want.abs() if dtype == torch.bfloat16 else 0.0)).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [40, 300])
def test_products_of_the_longest_contraction(dtype, rows):
    """K = 2^20: 16384 stages of a tile (300 rows: pairs of blocks)."""
    K, N = 1 << 20, 160
    x, W, status = whole((rows, K), -1, 1, 3), whole((1, N, K), 0, 1, 4), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ap.expert_linear(x, W, *one(rows), dtype=dtype, status=status).double()
    want = sum(a.double() @ b.double().t() for a, b in zip(x.split(1 << 17, 1), W[0].split(1 << 17, 1)))
    assert int(status) == 0
    assert bool(((got - want).abs() <= (HALF * want.abs() if dtype == torch.bfloat16 else 0.0)).all())
    # and back: a contraction over 2^20 features
    back = ap.expert_linear_dx(whole((rows, K), -1, 1, 5), whole((1, K, 72), 0, 1, 6), *one(rows), dtype=dtype, status=status).double()
    dy, V = whole((rows, K), -1, 1, 5), whole((1, K, 72), 0, 1, 6)[0]
    want = sum(a.double() @ b.double() for a, b in zip(dy.split(1 << 17, 1), V.split(1 << 17)))
    assert int(status) == 0
    assert bool(((back - want).abs() <= (HALF * want.abs() if dtype == torch.bfloat16 else 0.0)).all())


@pytest.mark.parametrize("N", [8, 200])
@pytest.mark.parametrize("seg,live", [([0, 10, 31], [10, 20, 30]), ([0, 10, -1], [10, 20, 30]), ([0, 10, 30], [10, 20, -4]),
                                      ([0, 10, 30], [10, 20, 2 ** 31 - 1]), ([0, 10, 30], [10, 20, 30])])
def test_bad_segments_of_the_bias_alone(N, seg, live):
    """The C call without dW says so too, and leaves their experts at 0."""
    import ctypes
    dy = whole((60, N), -3, 3, 1)
    s, n = to_dev(np.array(seg, np.int32)), to_dev(np.array(live, np.int32))
    db, status = torch.full((3, N), 7.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    at = [ctypes.c_void_p(t.data_ptr()) for t in (dy, s, n, db, status)]
    rc = ap.lib().ap_expert_linear_dw(at[0], N, None, 8, 60, 3, N, 8, at[1], at[2], 0, None, 2, at[3], None, 0, at[4],
                                      ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    good = live[2] == 30 and seg[2] == 30
    assert int(status) == (0 if good else ap.FLAG_BAD_COUNT)
    want = torch.stack([dy[:10].float().sum(0), dy[10:30].float().sum(0), dy[30:].float().sum(0) * good])
    assert torch.equal(db, want)


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("offset", [0, 3])
def test_bias_alone_from_python(add, offset):
    dy = whole((60, 96), -3, 3, 1)[:, offset:offset + 70]
    s, n = to_dev(np.array([0, 10, 30], np.int32)), to_dev(np.array([10, 0, 25], np.int32))
    db, status = torch.ones(3, 70, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    assert ap.expert_linear_dw(dy, None, s, n, dW=False, dbias=db, accumulate=add, status=status) is db
    want = torch.stack([dy[:10].float().sum(0), torch.zeros(70, device="cuda"), dy[30:55].float().sum(0)]) + (1.0 if add else 0.0)
    assert torch.equal(db, want) and int(status) == 0
    again = torch.ones(3, 70, device="cuda")
    ap.expert_linear_dw(dy, dy, s, n, dbias=again, accumulate=add, dW=torch.zeros(3, 70, 70, device="cuda"))
    assert torch.equal(db, again)
    for match, call in (("dbias", lambda: ap.expert_linear_dw(dy, None, s, n, dW=False)),
                        ("dbias must", lambda: ap.expert_linear_dw(dy, None, s, n, dW=False, dbias=db[:2]))):
        with pytest.raises(ValueError, match=match):
            call()


def section_bound(C):
    """FP32 results of a contraction of C places: sections of 1024 in the tensor cores, 17 x 2^-23 of the sum of magnitudes
    for each 16 places and once more, and a rounding for each section added up."""
    return (1024 / 16 + 1) * 17 * 2 * U + (C / 1024 + 1) * U


@pytest.mark.parametrize("live", [[200, 0, 90], [3, 1, 0], [700, 161, 33]])
@pytest.mark.parametrize("act", [None, "silu", "swiglu"])
@pytest.mark.parametrize("K", [65536, 8200])
def test_float_results_of_long_contractions(live, act, K):
    """Numbers of one sign, whose cut sums are all off the same way: at 65536 places by 3e-4 if they were added up in one."""
    E, N = len(live), 136 if K == 65536 else 300
    wide = 2 * N if act == "swiglu" else N
    seg = np.concatenate([[0], np.cumsum(live)[:-1] + 2]).astype(np.int32)
    n, rows = np.array(live, np.int32), int(sum(live)) + 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x = (torch.rand(rows, K, generator=g, device="cuda") + 0.5).bfloat16()
    W = (torch.rand(E, wide, K, generator=g, device="cuda") + 0.5).mul_(1 / K).bfloat16()
    res, bias = torch.randn(rows, N, generator=g, device="cuda").bfloat16(), torch.randn(E, wide, generator=g, device="cuda")
    out = ap.expert_linear(x, W, to_dev(seg), to_dev(n), bias=bias, act=act, residual=res, dtype=torch.float32,
                           out=torch.full((rows, N), 7.0, device="cuda"))
    again = ap.expert_linear(x, W, to_dev(seg), to_dev(n), bias=bias, act=act, residual=res, dtype=torch.float32,
                             out=torch.full((rows, N), 7.0, device="cuda"))
    assert torch.equal(out, again)
    back = ap.expert_linear_dx(x, W.transpose(1, 2).contiguous(), to_dev(seg), to_dev(n), dtype=torch.float32,
                               out=torch.full((rows, wide), 7.0, device="cuda"))
    on = np.zeros(rows, bool)
    for e, at in layer.expert_rows(seg, n, rows):
        on[torch.arange(rows).numpy()[at]] = True
        z = x[at].double() @ W[e].double().t()
        off = section_bound(K) * z  # (all terms are positive)
        assert bool(((back[at].double() - z).abs() <= off + U * z).all())
        b = bias[e].double()
        z, off = z + b, off + U * ((z + b).abs() + b.abs())
        if act == "swiglu":
            zg, zu, dg, du = z[:, :N], z[:, N:], off[:, :N], off[:, N:]
            want = torch.nn.functional.silu(zg) * zu
            # silu' <= 1.1, its own error (1.5 |z| + 12) u of itself
            off = 1.1 * dg * (zu.abs() + du) + zg.abs() * du + (1.5 * zg.abs() + 14) * U * want.abs()
        elif act == "silu":
            want = torch.nn.functional.silu(z)
            off = 1.1 * off + (1.5 * z.abs() + 12) * U * want.abs()
        else:
            want = z
        want = want + res[at].double()
        off = off + 2 * U * (want.abs() + res[at].double().abs())
        assert bool(((out[at].double() - want).abs() <= off).all())
    assert bool((out[torch.from_numpy(~on).cuda()] == 7.0).all()) and bool((back[torch.from_numpy(~on).cuda()] == 7.0).all())


def test_float_results_in_a_graph_and_on_another_stream():
    """Sections of a long contraction, with counts that change between replays."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x, W = torch.randn(600, 3000, generator=g, device="cuda").bfloat16(), torch.randn(2, 260, 3000, generator=g, device="cuda").bfloat16()
    seg, live = to_dev(np.array([0, 300], np.int32)), to_dev(np.array([300, 300], np.int32))
    out, side, graph = torch.empty(600, 130, device="cuda"), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        ap.expert_linear(x, W, seg, live, act="swiglu", out=out)
    for counts in ((300, 300), (1, 299), (0, 17), (257, 0)):
        live.copy_(torch.tensor(counts, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.full_like(out, 7.0)
        with torch.cuda.stream(side):
            ap.expert_linear(x, W, seg, live, act="swiglu", out=want, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert bool((out[counts[0]:300] == 7.0).all()) and bool((out[300 + counts[1]:] == 7.0).all())
        for e, n in enumerate(counts):
            z = x[300 * e:300 * e + n].double() @ W[e].double().t()
            size = x[300 * e:300 * e + n].double().abs() @ W[e].double().abs().t()
            off, zg, zu = section_bound(3000) * size, z[:, :130], z[:, 130:]
            h = torch.nn.functional.silu(zg)
            got = out[300 * e:300 * e + n].double()
            bound = 1.1 * off[:, :130] * (zu.abs() + off[:, 130:]) + h.abs() * off[:, 130:] + (1.5 * zg.abs() + 14) * U * (h * zu).abs()
            assert bool(((got - h * zu).abs() <= bound + 1e-30).all())
