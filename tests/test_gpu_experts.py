"""GPU parity: the experts' products and their gradients, against 64-bit plain
forms on the same BF16 operands.

Products of BF16 values are exact; the tensor cores add 16 of them to the FP32
accumulator at a time, each addend cut to the largest one's last bits: at most 17
x 2^-23 of the sum of magnitudes S a step, so (C / 16 + 1) 17 x 2^-23 S over a
contraction of C.  Bias and residual round by 2^-24 each (in S), 2^x and its
reciprocal make sigmoid good to (1.5 |z| + 8) 2^-24, the normal distribution's tail to
2e-7 + (0.75 z^2 + 4) 2^-24 of itself; a result
rounds by 2^-8 to BF16.  Errors of z reach the result through |act'| <= 1.13 (for
the gated product: times the other half, and the other way).
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
HALF = 2.0 ** -8


def chain(C):
    return (C / 16 + 1) * 17 * 2 * U


def f64(t):
    return t.detach().double().cpu().numpy()


class Rows:
    """Segments with gaps: `live` rows of each expert, `gap` unused rows (NaN) behind each."""

    def __init__(self, live, gap=0, seed=0, order=None):
        self.live = np.array(live, np.int32)
        E = len(live)
        seg, at = np.zeros(E, np.int32), 0
        for e in (range(E) if order is None else order):
            seg[e] = at
            at += int(self.live[e]) + gap
        self.seg, self.rows, self.E = seg, max(at, 1), E
        self.on = np.zeros(self.rows, bool)
        for _, s in layer.expert_rows(self.seg, self.live, self.rows):
            self.on[s] = True
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.args = to_dev(self.seg), to_dev(self.live)

    def make(self, cols, scale=1.0, pitch=None, offset=0, dtype=torch.bfloat16):
        """Rows of normal values, NaN where no expert has them, `pitch` apart, from element `offset` of their buffer on."""
        pitch = pitch or cols
        flat = torch.full((self.rows * pitch + offset + 8,), float("nan"), dtype=dtype, device="cuda")
        t = flat[offset:offset + self.rows * pitch].view(self.rows, pitch)[:, :cols]
        v = torch.randn(self.rows, cols, generator=self.g, device="cuda") * scale
        t.copy_(torch.where(to_dev(self.on)[:, None], v, float("nan")).to(dtype))
        return t

    def weights(self, N, K, offset=0, pitch=None, more=0):
        pitch = pitch or K
        flat = torch.full((self.E * (N * pitch + more) + offset + 8,), float("nan"), dtype=torch.bfloat16, device="cuda")
        t = flat[offset:].as_strided((self.E, N, K), (N * pitch + more, pitch, 1))
        t.copy_(torch.randn(self.E, N, K, generator=self.g, device="cuda") * K ** -0.5)
        return t


def zeros_off(a, on):
    return np.where(on[:, None], a, 0.0)


def check_forward(r, K, N, act=None, bias=False, residual=False, pre=True, dtype=torch.bfloat16, xo=0, xp=None, wo=0, wp=None,
                  more=0, out=None, op=None):
    wide = 2 * N if act == "swiglu" else N
    x, W = r.make(K, offset=xo, pitch=xp), r.weights(wide, K, wo, wp, more)
    b = torch.randn(r.E, wide, generator=r.g, device="cuda") if bias else None
    res = r.make(N, pitch=op) if residual else None
    out = torch.full((r.rows, op or N), 7.0, dtype=dtype, device="cuda")[:, :N]
    z = torch.full((r.rows, wide), 7.0, dtype=torch.bfloat16, device="cuda") if pre else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert ap.expert_linear(x, W, *r.args, bias=b, act=act, residual=res, out=out, pre=z, status=status) is out
    torch.cuda.synchronize()
    assert int(status) == 0
    ze, oe, size = layer.expert_linear(f64(x), f64(W), r.seg, r.live, None if b is None else f64(b), act,
                                       None if res is None else f64(res))
    got = f64(out)
    assert np.all(got[~r.on] == 7.0)
    dz = chain(K) * size + U * np.abs(ze)
    if pre:
        gz = f64(z)
        assert np.all(gz[~r.on] == 7.0)
        assert np.all((np.abs(gz - ze) <= dz + HALF * (np.abs(ze) + dz))[r.on])
    if act == "swiglu":
        g, u = ze[:, :N], ze[:, N:]
        s = (1.5 * np.abs(g) + 12) * U
        h = np.abs(layer.act("silu", g))
        bound = 1.13 * dz[:, :N] * (np.abs(u) + dz[:, N:]) + h * dz[:, N:] + s * h * np.abs(u)
    else:
        bound = 1.13 * dz + ((1.5 * np.abs(ze) + 12) * U + 2.0 ** -20) * np.abs(ze)
    bound = bound + 2 * U * (np.abs(oe) + (0 if res is None else np.abs(f64(res))))
    if dtype == torch.bfloat16:
        bound = bound + HALF * (np.abs(oe) + bound)
    assert np.all((np.abs(got - oe) <= bound + 1e-30)[r.on])
    return x, W, out


def check_rows(r, N, K, act=None, residual=False, dtype=torch.bfloat16, yo=0, yp=None, wo=0, wp=None):
    dy, W = r.make(N, offset=yo, pitch=yp), r.weights(N, K, wo, wp)
    wide = 2 * K if act == "swiglu" else K
    pre = r.make(wide) if act else None
    res = r.make(K) if residual else None
    out = torch.full((r.rows, wide), 7.0, dtype=dtype, device="cuda")
    ap.expert_linear_dx(dy, W, *r.args, act=act, pre=pre, residual=res, out=out)
    torch.cuda.synchronize()
    e, size = layer.expert_linear_dx(f64(dy), f64(W), r.seg, r.live, act, None if pre is None else f64(pre),
                                     None if res is None else f64(res))
    got = f64(out)
    assert np.all(got[~r.on] == 7.0)
    dd = (chain(N) + 2 * U) * size
    if act == "swiglu":
        z = np.abs(f64(pre))
        dd = np.concatenate([1.13 * dd * z[:, K:], dd * z[:, :K]], 1)
        z = np.concatenate([z[:, :K]] * 2, 1)
        size = np.concatenate([size, size], 1) * np.abs(np.concatenate([f64(pre)[:, K:], f64(pre)[:, :K]], 1))
    else:
        z = np.zeros_like(size) if act is None else np.abs(f64(pre))
        dd = 1.13 * dd
    # the slope's own terms (sigmoid, erfc, the density) do not exceed 1.5 + |z|; each within (3 |z| + 16) u or 2^-20
    bound = dd + (0 if act is None else ((3 * z + 16) * U + 2.0 ** -20) * (1.5 + z) * size) + 4 * U * np.abs(e)
    if dtype == torch.bfloat16:
        bound = bound + HALF * (np.abs(e) + bound)
    assert np.all((np.abs(got - e) <= bound + 1e-30)[r.on])


def check_weights(r, N, K, bias=True, add=False, dtype=torch.float32, yo=0, xo=0, yp=None, xp=None):
    dy, x = r.make(N, offset=yo, pitch=yp), r.make(K, offset=xo, pitch=xp)
    dW = torch.randn(r.E, N, K, generator=r.g, device="cuda").to(dtype)
    db = torch.randn(r.E, N, generator=r.g, device="cuda") if bias else None
    oldW, oldb = f64(dW), None if db is None else f64(db)
    ap.expert_linear_dw(dy, x, *r.args, dW=dW, dbias=db, accumulate=add)
    torch.cuda.synchronize()
    eW, eb, sW, sb = layer.expert_linear_dw(zeros_off(f64(dy), r.on), zeros_off(f64(x), r.on), r.seg, r.live, r.E)
    n = max(int(r.live.max()), 1)
    if add:
        eW, sW = eW + oldW, sW + np.abs(oldW)
    bound = (chain(n) + 2 * U) * sW
    if dtype == torch.bfloat16:
        bound = bound + HALF * (np.abs(eW) + bound)
    assert np.all(np.abs(f64(dW) - eW) <= bound)
    if bias:
        if add:
            eb, sb = eb + oldb, sb + np.abs(oldb)
        assert np.all(np.abs(f64(db) - eb) <= (n / 8 + 10) * U * sb)


RAGGED = [0, 1, 15, 16, 17, 0, 255, 256, 257, 31, 33, 300, 0]


def test_one_plain_product():
    check_forward(Rows([128]), 64, 128, pre=False)


def test_gelu_of_all_sizes():
    """z from -20 to 20 through a unit weight: the smaller tail within 2e-7 + (0.75 z^2 + 8) u of itself (below 2^-120: 0),
    the value z Phi(z) with one rounding more, 1 - tail another."""
    z = torch.linspace(-20, 20, 4001, device="cuda").bfloat16()
    n = z.numel()
    x = torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = z
    W = torch.zeros(1, 8, 8, dtype=torch.bfloat16, device="cuda")
    W[0, :, 0] = 1
    seg = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), n, dtype=torch.int32, device="cuda")
    f = f64(z)
    got = f64(ap.expert_linear(x, W, *seg, act="gelu", dtype=torch.float32))[:, 3]
    e = layer.act("gelu", f)
    tail = np.abs(f) * layer._cdf(-np.abs(f))
    rel = 2e-7 + (0.75 * f * f + 8) * U
    assert np.all(np.abs(got - e) <= rel * tail + 2 * U * np.abs(e) + 20 * 2.0 ** -120)
    pre = torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    pre[:, 0] = z
    dy = torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    dy[:, 0] = 1
    W = torch.zeros(1, 8, 8, dtype=torch.bfloat16, device="cuda")
    W[0, 0, :] = 1
    got = f64(ap.expert_linear_dx(dy, W, *seg, act="gelu", pre=pre, dtype=torch.float32))[:, 0]
    e = layer.act_backward("gelu", f, np.ones_like(f))
    bell = np.abs(f) * np.exp(-0.5 * f * f) / np.sqrt(2 * np.pi)
    assert np.all(np.abs(got - e) <= rel * (layer._cdf(-np.abs(f)) + 2 * bell) + 2 * U * np.abs(e) + 20 * 2.0 ** -120)


def test_one_product_of_a_gradient():
    check_rows(Rows([128]), 64, 128)


def test_one_product_of_a_pair_of_blocks():
    check_forward(Rows([256]), 64, 256, pre=False)


def test_one_product_of_a_gradient_by_a_pair_of_blocks():
    check_rows(Rows([256]), 64, 256)


def test_one_product_of_two_tiles_of_a_pair():
    check_forward(Rows([256]), 64, 512, pre=False)
    check_forward(Rows([200]), 64, 512, pre=False)


def test_one_product_of_a_gradient_by_two_tiles_of_a_pair():
    check_rows(Rows([256]), 64, 512)
    check_rows(Rows([30, 300]), 64, 512)


def test_one_gradient_of_weights():
    check_weights(Rows([64]), 128, 64, bias=False)


@pytest.mark.parametrize("K,N", [(64, 128), (256, 384), (8, 8), (72, 200), (1000, 136), (2048, 264)])
@pytest.mark.parametrize("act", [None, "silu", "gelu", "swiglu"])
def test_forward(K, N, act):
    check_forward(Rows(RAGGED, gap=3), K, N, act, bias=True, residual=True)


@pytest.mark.parametrize("N", [8, 15, 16, 17, 24, 32, 48, 64])
@pytest.mark.parametrize("residual", [True, False])
def test_gated_halves_of_any_width(N, residual):
    """Widths at which a writer's 16 features of either half end."""
    check_forward(Rows([40, 3]), 64, N, "swiglu", bias=True, residual=residual)
    check_rows(Rows([40, 3]), 64, N, "swiglu", residual=residual)


MANY = [0, 1, 31, 32, 33, 255, 256, 257, 511, 513, 700, 16, 17, 0]


@pytest.mark.parametrize("K,N", [(64, 136), (256, 384), (72, 200), (1000, 264), (520, 1000), (512, 640)])
@pytest.mark.parametrize("act", [None, "silu", "swiglu"])
def test_many_rows(K, N, act):
    """Tiles of 256 rows, shared out evenly; pairs of blocks."""
    r = Rows(MANY, gap=2)
    check_forward(r, K, N, act, bias=True, residual=True)
    check_rows(r, K, N, act, residual=True)
    check_weights(r, N, K, False)


@pytest.mark.parametrize("K,N", [(1, 1), (63, 65), (65, 127), (203, 517), (1003, 130)])
@pytest.mark.parametrize("act", [None, "gelu", "swiglu"])
def test_forward_of_odd_rows(K, N, act):
    check_forward(Rows([3, 0, 130, 257, 1], gap=1), K, N, act, bias=True, residual=True)


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forward_types_pitches_and_offsets(act, dtype):
    r = Rows([40, 0, 300], gap=2)
    check_forward(r, 96, 72, act, dtype=dtype)
    check_forward(r, 96, 72, act, dtype=dtype, xp=104, wp=112, more=16, op=75)  # rows apart, still by tensor map
    check_forward(r, 99, 72, act, dtype=dtype, xp=104, wp=112)                  # odd rows at even pitches
    check_forward(r, 96, 72, act, dtype=dtype, xo=1)                            # between 16-byte boundaries
    check_forward(r, 96, 72, act, dtype=dtype, wo=3)
    check_forward(r, 96, 72, act, dtype=dtype, xp=97)
    check_forward(r, 96, 72, act, pre=False, dtype=dtype)


@pytest.mark.parametrize("live", [[1], [4] * 5, [700], [2000, 1], [90] * 3, [0, 0], [30] * 40])
@pytest.mark.parametrize("K,N", [(320, 192), (101, 70)])
def test_numbers_of_rows(live, K, N):
    """Tiles of 64, 128 and 256 rows, chosen by the average; one token's few rows."""
    r = Rows(live)
    check_forward(r, K, N, "swiglu")
    check_rows(r, K, N, "swiglu")
    check_weights(r, N, K)


def test_more_experts_than_a_block_has_lanes():
    live = inputs.rng(3, 3).integers(0, 6, 1024)
    r = Rows(live, gap=1, order=inputs.rng(4, 3).permutation(1024))
    check_forward(r, 32, 24, "silu")
    check_rows(r, 32, 24, "silu")
    check_weights(r, 24, 32)


def test_long_contractions():
    """More stages than the ring has, several times over."""
    r = Rows([50, 200])
    check_forward(r, 8192, 128, pre=False)
    check_rows(r, 8192, 128)
    check_weights(Rows([5000, 64, 65]), 128, 256)


@pytest.mark.parametrize("add", [True, False])
@pytest.mark.parametrize("N,K", [(128, 256), (130, 67)])
def test_long_sums_of_weights(N, K, add):
    """FP32 gradients are added up by sections of 2048 rows: an error of 1.1e-9 of the result for each row of a section,
    and for numbers of one sign (each addition cuts up to 2 u of the sum so far, half of it on the average) up to
    2048 / 16 u = 128 u, whatever the number of rows; additions of sections round by u each."""
    r = Rows([2048, 9000, 0, 2049, 4096])
    for positive in (False, True):
        x, dy = r.make(K), r.make(N)
        if positive:
            x, dy = x.abs(), dy.abs()
        dW = torch.ones(r.E, N, K, device="cuda")
        ap.expert_linear_dw(dy, x, *r.args, dW=dW, accumulate=add)
        e, _, _, _ = layer.expert_linear_dw(f64(dy), f64(x), r.seg, r.live, r.E)
        e = e + (1.0 if add else 0.0)
        for q in range(r.E):
            size = np.linalg.norm(e[q])
            assert np.linalg.norm(f64(dW[q]) - e[q]) <= ((128 + 8) * U if positive else 4e-6) * size


@pytest.mark.parametrize("N,K", [(64, 128), (256, 384), (8, 8), (72, 200), (1000, 136)])
@pytest.mark.parametrize("act", [None, "silu", "gelu", "swiglu"])
def test_gradient_of_rows(N, K, act):
    check_rows(Rows(RAGGED, gap=3), N, K, act, residual=True)


@pytest.mark.parametrize("N,K", [(1, 1), (63, 65), (203, 131)])
@pytest.mark.parametrize("act", [None, "gelu", "swiglu"])
def test_gradient_of_odd_rows(N, K, act):
    check_rows(Rows([3, 0, 130, 257, 1], gap=1), N, K, act, residual=True)
    check_rows(Rows([3, 130]), 64, 72, act, yo=1, dtype=torch.float32)
    check_rows(Rows([3, 130]), 64, 72, act, wp=75)


@pytest.mark.parametrize("N,K", [(64, 128), (256, 384), (8, 8), (72, 200), (136, 1000), (130, 514)])
@pytest.mark.parametrize("add", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_of_weights(N, K, add, dtype):
    check_weights(Rows(RAGGED, gap=3), N, K, True, add, dtype)


@pytest.mark.parametrize("N,K", [(1, 1), (63, 65), (131, 203)])
@pytest.mark.parametrize("add", [True, False])
def test_gradient_of_odd_weights(N, K, add):
    check_weights(Rows([3, 0, 130, 257, 1], gap=1), N, K, True, add)
    check_weights(Rows([3, 130]), 64, 72, yo=1, add=add)
    check_weights(Rows([3, 130]), 64, 72, xp=73, add=add, dtype=torch.bfloat16)


@pytest.mark.parametrize("N", [8, 64, 100, 128, 130, 512])
@pytest.mark.parametrize("add", [True, False])
def test_gradient_of_the_bias_alone(N, add):
    """The C call without dW: the same sums up to their order."""
    import ctypes
    r = Rows(RAGGED, gap=2)
    dy = r.make(N)
    db = torch.randn(r.E, N, generator=r.g, device="cuda")
    old = f64(db)
    rc = ap.lib().ap_expert_linear_dw(ctypes.c_void_p(dy.data_ptr()), N, None, 8, r.rows, r.E, N, 8, ctypes.c_void_p(r.args[0].data_ptr()),
                                      ctypes.c_void_p(r.args[1].data_ptr()), int(add), None, 2, ctypes.c_void_p(db.data_ptr()), None, 0,
                                      None, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    _, e, _, size = layer.expert_linear_dw(zeros_off(f64(dy), r.on), np.zeros((r.rows, 8)), r.seg, r.live, r.E)
    if add:
        e, size = e + old, size + np.abs(old)
    assert np.all(np.abs(f64(db) - e) <= (300 / 8 + 10) * U * size)


def test_neighbours_do_not_leak():
    """NaN in another expert's weights and rows, and in rows of no expert, stays there."""
    for K in (96, 99):
        r = Rows([70, 5, 64, 100], gap=0)
        x, W = r.make(K), r.weights(64, K)
        a = ap.expert_linear(x, W, *r.args, act="gelu")
        d = ap.expert_linear_dx(a, W, *r.args)
        w = ap.expert_linear_dw(a, x, *r.args)
        x2, W2 = x.clone(), W.clone()
        x2[70:75] = float("nan")
        W2[1] = float("inf")
        a2 = a.clone()
        a2[70:75] = float("nan")
        b = ap.expert_linear(x2, W2, *r.args, act="gelu")
        d2 = ap.expert_linear_dx(a2, W2, *r.args)
        w2 = ap.expert_linear_dw(a2, x2, *r.args)
        for p, q in ((a, b), (d, d2)):
            assert torch.equal(p[:70], q[:70]) and torch.equal(p[75:], q[75:])
            assert q[70:75].isnan().all()
        assert all(torch.equal(w[e], w2[e]) for e in (0, 2, 3)) and w2[1].isnan().all()


def test_bad_segments_are_left_out():
    r = Rows([10, 20, 30], gap=0)
    x, W = r.make(64), r.weights(64, 64)
    good = ap.expert_linear(x, W, *r.args)
    for seg, live in (([0, 10, 31], [10, 20, 30]), ([0, 10, -1], [10, 20, 30]), ([0, 10, 30], [10, 20, -4]),
                      ([0, 10, 30], [10, 20, 2 ** 31 - 1])):
        s, n = to_dev(np.array(seg, np.int32)), to_dev(np.array(live, np.int32))
        for call in (lambda st, o: ap.expert_linear(x, W, s, n, out=o, status=st),
                     lambda st, o: ap.expert_linear_dx(x, W, s, n, out=o, status=st)):
            status, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((60, 64), 7.0, dtype=torch.bfloat16, device="cuda")
            call(status, out)
            assert int(status) == ap.FLAG_BAD_COUNT
            assert bool((out[30:] == 7.0).all())
        out = ap.expert_linear(x, W, s, n)
        assert torch.equal(out[:30], good[:30])
        status, db = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones(3, 64, device="cuda")
        dW = ap.expert_linear_dw(x, x, s, n, dbias=db, status=status)
        assert int(status) == ap.FLAG_BAD_COUNT and not dW[2].any() and not db[2].any() and bool(dW[0].any())


def test_in_place():
    r = Rows([10, 200], gap=1)
    x, W, z = r.make(64), r.weights(128, 64), r.make(128)
    res = r.make(128)
    kept = res.clone()
    a = ap.expert_linear(x, W, *r.args, residual=kept, out=torch.zeros_like(res))
    ap.expert_linear(x, W, *r.args, residual=res, out=res)
    on = to_dev(r.on)
    assert torch.equal(a[on], res[on])
    dy, V = r.make(96), r.weights(96, 64)
    g = ap.expert_linear_dx(dy, V, *r.args, act="swiglu", pre=z)
    ap.expert_linear_dx(dy, V, *r.args, act="swiglu", pre=z, out=z)
    assert torch.equal(g[on], z[on])


def test_gradients_against_differences():
    """The chain of both products and a gate: the loss's differences along a direction of every input."""
    r = Rows([5, 9, 0, 3])
    H, F = 16, 24
    x, W1, W2 = r.make(H, 0.5), r.weights(2 * F, H), r.weights(H, F)
    dy = r.make(H)
    z = torch.empty(r.rows, 2 * F, dtype=torch.bfloat16, device="cuda")
    h = ap.expert_linear(x, W1, *r.args, act="swiglu", pre=z)
    dz = ap.expert_linear_dx(dy, W2, *r.args, act="swiglu", pre=z)
    dx = ap.expert_linear_dx(dz, W1, *r.args, dtype=torch.float32)
    g1, g2 = ap.expert_linear_dw(dz, x, *r.args), ap.expert_linear_dw(dy, h, *r.args)

    def loss(x, a, b):
        _, y, _ = layer.expert_linear(x, a, r.seg, r.live, None, "swiglu")
        _, o, _ = layer.expert_linear(y, b, r.seg, r.live)
        return float((o * f64(dy)).sum())
    v, step = [f64(t) for t in (x, W1, W2)], 1e-5
    for q, g in enumerate((dx, g1, g2)):
        d = inputs.rng(q, 7).standard_normal(v[q].shape)
        ends = []
        for sign in (1, -1):
            w = list(v)
            w[q] = w[q] + sign * step * d
            ends.append(loss(*w))
        slope = (ends[0] - ends[1]) / (2 * step)
        # z, h and dz were rounded to BF16: three roundings of 2^-8 along the longest path of each term
        assert abs((f64(g) * d).sum() - slope) <= 3 * HALF * np.abs(f64(g) * d).sum()


def test_captured_and_replayed_with_new_counts():
    E, K, N = 6, 128, 160
    r = Rows([40] * E)
    x, W = r.make(K), r.weights(N, K)
    seg, live = r.args
    out, dx = torch.zeros(r.rows, N, dtype=torch.bfloat16, device="cuda"), torch.zeros(r.rows, K, dtype=torch.bfloat16, device="cuda")
    dW = torch.zeros(E, N, K, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ap.expert_linear(x, W, seg, live, act="silu", out=out)
        ap.expert_linear_dx(out, W, seg, live, out=dx)
        ap.expert_linear_dw(out, x, seg, live, dW=dW)
    for counts in ([40] * E, [0, 100, 3, 80, 1, 56], [240, 0, 0, 0, 0, 0], [0] * E):
        live.copy_(torch.tensor(counts, dtype=torch.int32))
        seg.copy_(live.cumsum(0) - live)
        out.zero_(), dx.zero_()
        g.replay()
        torch.cuda.synchronize()
        o2 = ap.expert_linear(x, W, seg, live, act="silu", out=torch.zeros_like(out))
        assert torch.equal(out, o2)
        assert torch.equal(dx, ap.expert_linear_dx(o2, W, seg, live, out=torch.zeros_like(dx)))
        assert torch.equal(dW, ap.expert_linear_dw(o2, x, seg, live))
        _, e, size = layer.expert_linear(f64(x), f64(W), host(seg), host(live), None, "silu")
        on = ~np.isnan(e[:, 0])
        assert np.all((np.abs(f64(out) - e) <= 1.13 * chain(K) * size + 1.1 * HALF * np.abs(e) + 1e-6)[on])


def test_equal_inputs_equal_bits_on_any_stream():
    r = Rows([513, 3, 900, 64])
    x, W, dy = r.make(512), r.weights(640, 512), r.make(640)
    first = None
    for q in range(6):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = (ap.expert_linear(x, W, *r.args, act="gelu", stream=s), ap.expert_linear_dx(dy, W, *r.args, stream=s),
               ap.expert_linear_dw(dy, x, *r.args, stream=s))
        torch.cuda.synchronize()
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_no_rows():
    W = torch.zeros(3, 8, 16, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    assert ap.expert_linear(x, W, none, none).shape == (0, 8)
    dy = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
    assert ap.expert_linear_dx(dy, W, none, none).shape == (0, 16)
    dW, db = torch.ones(3, 8, 16, device="cuda"), torch.ones(3, 8, device="cuda")
    ap.expert_linear_dw(dy, x, none, none, dW=dW, dbias=db, accumulate=True)
    assert bool((dW == 1).all()) and bool((db == 1).all())
    ap.expert_linear_dw(dy, x, none, none, dW=dW, dbias=db)
    assert not dW.any() and not db.any()


def test_refusals():
    x = torch.zeros(10, 16, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(2, 8, 16, dtype=torch.bfloat16, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    y = torch.zeros(10, 8, dtype=torch.bfloat16, device="cuda")
    for match, call in (
            ("act", lambda: ap.expert_linear(x, W, n, n, act="relu")),
            ("bfloat16", lambda: ap.expert_linear(x.float(), W, n, n)),
            ("W must", lambda: ap.expert_linear(x, W.float(), n, n)),
            ("W must", lambda: ap.expert_linear(x, W[0], n, n)),
            ("W must", lambda: ap.expert_linear(x, W.transpose(1, 2), n, n)),
            ("x must", lambda: ap.expert_linear(x[:, :8], W, n, n)),
            ("live", lambda: ap.expert_linear(x, W, n, n[:1])),
            ("seg_off", lambda: ap.expert_linear(x, W, n.long(), n)),
            ("bias", lambda: ap.expert_linear(x, W, n, n, bias=torch.zeros(2, 8, dtype=torch.bfloat16, device="cuda"))),
            ("even", lambda: ap.expert_linear(x, W[:, :7], n, n, act="swiglu")),
            ("residual", lambda: ap.expert_linear(x, W, n, n, residual=x)),
            ("pre", lambda: ap.expert_linear(x, W, n, n, pre=x)),
            ("out", lambda: ap.expert_linear(x, W, n, n, out=x)),
            ("dtype", lambda: ap.expert_linear(x, W, n, n, dtype=torch.float16)),
            ("pre", lambda: ap.expert_linear_dx(y, W, n, n, act="silu")),
            ("pre", lambda: ap.expert_linear_dx(y, W, n, n, act="swiglu", pre=x)),
            ("dy", lambda: ap.expert_linear_dx(x, W, n, n)),
            ("accumulate", lambda: ap.expert_linear_dw(y, x, n, n, accumulate=True)),
            ("dW", lambda: ap.expert_linear_dw(y, x, n, n, dW=torch.zeros(2, 16, 8, device="cuda"))),
            ("dbias", lambda: ap.expert_linear_dw(y, x, n, n, dbias=torch.zeros(2, 9, device="cuda"))),
            ("status", lambda: ap.expert_linear(x, W, n, n, status=torch.zeros(1)))):
        with pytest.raises(ValueError, match=match):
            call()


@pytest.mark.parametrize("sms", [8, 24])
def test_on_partitions(sms):
    """Streams of SM partitions, which take fewer pairs of blocks or none: the bits of an ordinary stream."""
    import ctypes
    from activation_paging_gb300 import build as cuda_build
    lib = ctypes.CDLL(cuda_build.BENCH_LIB)
    vp, ip = ctypes.c_void_p, ctypes.c_int
    s1, s2, c1, c2, n1, n2 = vp(), vp(), vp(), vp(), ip(), ip()
    lib.apb_green_split.restype = ip
    lib.apb_green_split.argtypes = [ip, ip] + [ctypes.POINTER(vp)] * 2 + [ctypes.POINTER(ip)] * 2 + [ctypes.POINTER(vp)] * 2
    lib.apb_green_destroy.restype = ip
    lib.apb_green_destroy.argtypes = [vp] * 4
    rc = lib.apb_green_split(torch.cuda.current_device(), sms, *(ctypes.byref(t) for t in (s1, s2, n1, n2, c1, c2)))
    if rc < 0:
        pytest.skip(f"the driver lacks green-context entry point {-rc} of apb_green_split")
    assert rc == 0
    r = Rows([513, 3, 900, 64])
    x, W, dy, z = r.make(256), r.weights(512, 256), r.make(512), r.make(512)
    logits = torch.randn(3000, 64, generator=r.g, device="cuda")

    def calls():
        return [ap.expert_linear(x, W, *r.args, act="swiglu"), ap.expert_linear_dx(dy, W, *r.args, act="swiglu", pre=z),
                ap.expert_linear_dw(dy, x, *r.args), *ap.route_scored(logits, 8, groups=8, top_groups=4)]
    first = calls()
    for h in (s1, s2):
        s = torch.cuda.ExternalStream(h.value)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = calls()
        torch.cuda.synchronize()
        for a, b in zip(first, got):
            assert torch.equal(a, b)  # (every row is some expert's)
    torch.cuda.synchronize()
    assert lib.apb_green_destroy(s1, s2, c1, c2) == 0
