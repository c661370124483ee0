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
