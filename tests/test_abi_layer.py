"""Routing by scores, the experts' products and the weights' update reject bad
arguments on the host, before any launch (no GPU is touched)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from activation_paging_gb300 import build, _lib
    build.build()
    return _lib.load()


P = ctypes.c_void_p(4096)


def test_route_scored_refusals(lib):
    def call(logits=P, T=100, E=64, k=8, score=1, bias=None, groups=8, top=4, best=2, idx=P, w=P):
        return lib.ap_route_scored(logits, T, E, k, score, bias, groups, top, best, 1, 1.0, None, idx, w, None, None)
    n0 = lib.ap_launch_count()
    for bad in (dict(E=0), dict(E=1025), dict(k=0), dict(k=33, E=64, groups=1, top=1), dict(k=65), dict(T=-1), dict(T=2 ** 31),
                dict(score=2), dict(score=-1), dict(groups=0), dict(groups=33, E=66), dict(groups=7), dict(top=0), dict(top=9),
                dict(groups=16, top=1), dict(best=0), dict(best=3), dict(E=32, groups=32, top=8), dict(logits=None),
                dict(idx=None), dict(w=None)):
        assert call(**bad) == -1, bad
    assert call(T=0, logits=None, idx=None, w=None) == 0
    assert lib.ap_launch_count() == n0


def test_route_scored_backward_refusals(lib):
    def call(logits=P, T=10, E=16, k=2, idx=P, dw=P, score=0, d=P):
        return lib.ap_route_scored_backward(logits, T, E, k, idx, dw, score, 1, 1.0, d, None, None)
    n0 = lib.ap_launch_count()
    for bad in (dict(E=0), dict(k=17), dict(T=-1), dict(score=5), dict(logits=None), dict(idx=None), dict(dw=None), dict(d=None)):
        assert call(**bad) == -1, bad
    assert call(T=0, logits=None, idx=None, dw=None, d=None) == 0
    assert lib.ap_launch_count() == n0


def test_route_bias_step_refusals(lib):
    n0 = lib.ap_launch_count()
    assert lib.ap_route_bias_step(P, P, 0, 1.0, 0, None) == -1
    assert lib.ap_route_bias_step(P, P, 1025, 1.0, 0, None) == -1
    assert lib.ap_route_bias_step(None, P, 8, 1.0, 0, None) == -1
    assert lib.ap_route_bias_step(P, None, 8, 1.0, 0, None) == -1
    assert lib.ap_launch_count() == n0


def adamw(lib, tensor=(), **over):
    from activation_paging_gb300._lib import AdamWConfig, AdamWTensor
    t = (AdamWTensor * 2)()
    for e in t:
        e.param = e.grad = e.master = e.m = e.v = e.m_scale = e.v_scale = 4096
        e.n = 1000
    for name, value in tensor:
        setattr(t[1], name, value)
    c = AdamWConfig(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, param_dtype=0, grad_dtype=2, master=1, state_bits=8, d_step=4096)
    n = over.pop("n", 2)
    for name, value in over.items():
        setattr(c, name, value)
    return lib.ap_adamw_step(t, n, ctypes.byref(c), None)


def test_adamw_step_refusals(lib):
    n0 = lib.ap_launch_count()
    for over in (dict(n=-1), dict(param_dtype=1), dict(grad_dtype=3), dict(state_bits=16), dict(master=2),
                 dict(param_dtype=2), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(beta1=float("nan")),
                 dict(d_step=0), dict(d_step=4098)):
        assert adamw(lib, **over) == -1, over
    for name in ("param", "grad", "master", "m", "v", "m_scale", "v_scale"):
        assert adamw(lib, [(name, 0)]) == -1, name
        assert adamw(lib, [(name, 4097)]) == -1, name
    assert adamw(lib, [("n", -5)]) == -1
    assert adamw(lib, [("n", 2 ** 39)]) == -1
    assert lib.ap_adamw_step(None, 0, None, None) == -1
    assert lib.ap_launch_count() == n0


def test_grad_norm_refusals(lib):
    from activation_paging_gb300._lib import AdamWTensor
    t = (AdamWTensor * 2)()
    for e in t:
        e.grad, e.n = 4096, 1000
    n = ctypes.c_int64()
    assert lib.ap_grad_norm_scratch_bytes(t, 2, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.ap_grad_norm_scratch_bytes(t, 2, None) == -1
    n0 = lib.ap_launch_count()

    def call(tensors=t, count=2, dtype=2, out=P, scratch=P, sb=n.value):
        return lib.ap_grad_norm(tensors, count, dtype, 1.0, out, scratch, sb, None)
    for bad in (dict(count=-1), dict(tensors=None), dict(dtype=1), dict(out=None), dict(scratch=None), dict(sb=n.value - 1),
                dict(scratch=ctypes.c_void_p(4100))):
        assert call(**bad) == -1, bad
    t[1].grad = 4098
    assert call() == -1
    t[1].grad = 0
    assert call() == -1
    assert lib.ap_launch_count() == n0


def test_adamw_moments_refusals(lib):
    def call(m=P, v=P, ms=P, vs=P, n=512, dtype=0, mo=P, vo=P):
        return lib.ap_adamw_moments(m, v, ms, vs, n, dtype, mo, vo, None)
    n0 = lib.ap_launch_count()
    for bad in (dict(n=-256), dict(n=100), dict(dtype=1), dict(m=None), dict(v=None), dict(ms=None), dict(vs=None), dict(mo=None),
                dict(vo=None), dict(m=ctypes.c_void_p(4097)), dict(mo=ctypes.c_void_p(4100))):
        assert call(**bad) == -1, bad
    assert call(n=0, m=None) == 0
    assert lib.ap_launch_count() == n0


def test_expert_linear_refusals(lib):
    def fwd(x=P, ldx=64, rows=100, E=4, N=32, K=64, seg=P, live=P, W=P, ldw=64, lde=64 * 64, bias=None, act=0, res=None, ldr=32,
            pre=None, ldp=32, out=P, ldo=32, dt=0, scratch=None, sb=0):
        return lib.ap_expert_linear(x, ldx, rows, E, N, K, seg, live, W, ldw, lde, bias, act, res, ldr, pre, ldp, out, ldo, dt, scratch,
                                    sb, None, None)
    odd, half = ctypes.c_void_p(4097), ctypes.c_void_p(4098)
    n0 = lib.ap_launch_count()
    for bad in (dict(rows=-1), dict(rows=2 ** 31), dict(E=0), dict(E=1025), dict(N=0), dict(K=0), dict(N=2 ** 20 + 1), dict(K=2 ** 21),
                dict(ldx=63), dict(ldw=63), dict(lde=31 * 64), dict(act=4), dict(act=-1), dict(act=3, lde=63 * 64), dict(dt=1), dict(ldo=31),
                dict(res=P, ldr=31), dict(pre=P, ldp=31), dict(act=3, pre=P, ldp=63), dict(x=None), dict(seg=None), dict(live=None),
                dict(W=None), dict(out=None), dict(x=odd), dict(W=odd), dict(out=odd), dict(res=odd), dict(pre=odd), dict(bias=half),
                dict(dt=2, out=half), dict(rows=2 ** 31 - 1, N=2 ** 20, ldo=2 ** 20, lde=2 ** 27, ldw=64)):
        assert fwd(**bad) == -1, bad
    assert fwd(rows=0, x=None, out=None) == 0
    # operands off the 16-byte boundaries need work space
    n = ctypes.c_int64(-1)
    assert lib.ap_expert_linear_scratch_bytes(P, 64, 100, 64, P, 64, 4096, 128, 64, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.ap_expert_linear_scratch_bytes(P, 65, 100, 63, P, 64, 4096, 128, 64, ctypes.byref(n)) == 0
    assert n.value == 100 * 128
    assert lib.ap_expert_linear_scratch_bytes(half, 64, 100, 64, P, 64, 4097, 128, 63, ctypes.byref(n)) == 0
    assert n.value == 100 * 128 + 128 * 128
    assert lib.ap_expert_linear_scratch_bytes(P, 64, -1, 64, P, 64, 0, 128, 64, ctypes.byref(n)) == -1
    assert lib.ap_expert_linear_scratch_bytes(P, 64, 1, 0, P, 64, 0, 128, 64, ctypes.byref(n)) == -1
    assert lib.ap_expert_linear_scratch_bytes(P, 64, 1, 64, P, 64, 0, 128, 64, None) == -1
    for bad in (dict(x=half), dict(ldx=65), dict(W=half), dict(ldw=65, lde=4224), dict(x=half, scratch=P, sb=100 * 128 - 1),
                dict(x=half, scratch=ctypes.c_void_p(4104), sb=100 * 128)):
        assert fwd(**bad) == -1, bad
        assert b"scratch" in lib.ap_last_error()

    def dx(dy=P, ldy=32, rows=100, E=4, N=32, K=64, seg=P, live=P, W=P, ldw=64, lde=32 * 64, act=0, pre=None, ldp=64, res=None, ldr=64,
           out=P, ldo=64, dt=0):
        return lib.ap_expert_linear_dx(dy, ldy, rows, E, N, K, seg, live, W, ldw, lde, act, pre, ldp, res, ldr, out, ldo, dt, None, 0,
                                       None, None)
    for bad in (dict(rows=-1), dict(E=0), dict(ldy=31), dict(ldw=63), dict(lde=30 * 64), dict(act=1), dict(act=3, pre=P, ldp=127, ldo=128),
                dict(act=3, pre=P, ldp=128), dict(res=P, ldr=63), dict(dt=1), dict(dy=None), dict(out=None), dict(act=9)):
        assert dx(**bad) == -1, bad

    def dw(dy=P, ldy=32, x=P, ldx=64, rows=100, E=4, N=32, K=64, seg=P, live=P, add=0, dW=P, dt=2, db=None):
        return lib.ap_expert_linear_dw(dy, ldy, x, ldx, rows, E, N, K, seg, live, add, dW, dt, db, None, 0, None, None)
    for bad in (dict(rows=-1), dict(E=1025), dict(ldy=31), dict(ldx=63), dict(add=2), dict(dt=1), dict(dW=None), dict(dy=None),
                dict(x=None), dict(seg=None), dict(live=None), dict(dW=half), dict(db=half), dict(x=odd)):
        assert dw(**bad) == -1, bad
    assert lib.ap_launch_count() == n0
