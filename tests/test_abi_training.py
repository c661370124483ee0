"""The training operators reject bad arguments on the host, before any launch
(no GPU is touched), and their work-space sizes grow as documented."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from activation_paging_gb300 import build, _lib
    build.build()
    return _lib.load()


P = ctypes.c_void_p(4096)


def test_route_balance_refusals(lib):
    n = ctypes.c_int64()
    assert lib.ap_route_balance_scratch_bytes(5000, 128, 0, ctypes.byref(n)) == 0

    def call(logits=P, T=5000, E=128, k=8, S=0, mask=None, idx=P, w=P, counts=P, prob=P, slope=P, loss=P, scratch=P,
             sb=n.value):
        return lib.ap_route_balance(logits, T, E, k, S, mask, 0.01, idx, w, counts, prob, slope, loss, scratch, sb,
                                    None)
    n0 = lib.ap_launch_count()
    assert call(E=0) == -1
    assert call(E=1025) == -1
    assert call(k=0) == -1
    assert call(k=33) == -1
    assert call(E=4, k=5) == -1
    assert call(T=-1) == -1
    assert call(T=2 ** 31) == -1
    assert call(S=-1) == -1
    for name in ("logits", "idx", "w", "counts", "prob", "slope", "loss", "scratch"):
        assert call(**{name: None}) == -1, name
    assert b"NULL" in lib.ap_last_error()
    assert call(sb=n.value - 1) == -1
    assert b"scratch" in lib.ap_last_error()
    assert call(scratch=ctypes.c_void_p(4096 + 4)) == -1
    assert call(T=0, loss=None) == -1
    assert call(T=2 ** 31 - 1, E=1024, S=1, sb=2 ** 62) == -1  # more groups than one launch takes
    assert lib.ap_launch_count() == n0


def test_route_backward_refusals(lib):
    def call(logits=P, T=10, E=16, k=2, idx=P, w=P, dw=P, slope=P, dloss=None, S=0, dlogits=P):
        return lib.ap_route_backward(logits, T, E, k, idx, w, dw, slope, dloss, S, None, dlogits, None, None)
    n0 = lib.ap_launch_count()
    assert call(E=0) == -1
    assert call(k=17) == -1
    assert call(T=-1) == -1
    assert call(S=-2) == -1
    assert call(dlogits=None) == -1
    assert call(idx=None) == -1
    assert call(w=None) == -1
    assert call(logits=None) == -1
    assert call(T=0, logits=None, idx=None, w=None, dw=None, slope=None, dlogits=None) == 0
    assert lib.ap_launch_count() == n0


def test_embed_refusals(lib):
    def call(table=P, V=100, tld=64, tt=0, ids=P, ib=8, T=10, H=64, out=P, old=64, ot=0):
        return lib.ap_embed(table, V, tld, tt, ids, ib, T, H, 1.0, out, old, ot, None, None)
    n0 = lib.ap_launch_count()
    assert call(V=0) == -1
    assert call(V=2 ** 31) == -1
    assert call(H=0) == -1
    assert call(T=-1) == -1
    assert call(tld=63) == -1
    assert call(old=63) == -1
    assert call(tt=1) == -1   # no E4M3 tables
    assert call(ot=3) == -1
    assert call(ib=2) == -1
    assert call(table=None) == -1
    assert call(ids=None) == -1
    assert call(out=None) == -1
    assert call(table=ctypes.c_void_p(4097)) == -1
    assert call(ids=ctypes.c_void_p(4100)) == -1
    assert call(ot=2, out=ctypes.c_void_p(4098)) == -1
    assert call(T=0, table=None, ids=None, out=None) == 0
    assert lib.ap_launch_count() == n0


def test_embed_backward_refusals(lib):
    n = ctypes.c_int64()
    assert lib.ap_embed_scratch_bytes(5000, 5000, 64, ctypes.byref(n)) == 0

    def call(dout=P, dld=64, dt=0, ids=P, ib=4, T=5000, H=64, V=5000, pad=-1, acc=0, dtable=P, gld=64, gt=2, scratch=P,
             sb=n.value):
        return lib.ap_embed_backward(dout, dld, dt, ids, ib, T, H, V, pad, 1.0, acc, dtable, gld, gt, scratch, sb,
                                     None, None)
    n0 = lib.ap_launch_count()
    assert call(H=0) == -1
    assert call(V=0) == -1
    assert call(T=2 ** 31) == -1
    assert call(dld=60) == -1
    assert call(gld=60) == -1
    assert call(pad=-2) == -1
    assert call(pad=5000) == -1
    assert call(dt=1) == -1
    assert call(gt=1) == -1
    assert call(ib=3) == -1
    assert call(acc=2) == -1
    for name in ("dout", "ids", "dtable", "scratch"):
        assert call(**{name: None}) == -1, name
    assert call(sb=n.value - 1) == -1
    assert call(scratch=ctypes.c_void_p(4096 + 8)) == -1
    assert call(dtable=ctypes.c_void_p(4098)) == -1
    assert call(T=0, acc=1, dout=None, ids=None, dtable=None, scratch=None) == 0
    assert call(T=0, acc=0, dtable=None) == -1
    assert lib.ap_launch_count() == n0


def test_scratch_sizes(lib):
    n = ctypes.c_int64()

    def balance(T, E, S):
        assert lib.ap_route_balance_scratch_bytes(T, E, S, ctypes.byref(n)) == 0
        return n.value

    def emb(T, V, H):
        assert lib.ap_embed_scratch_bytes(T, V, H, ctypes.byref(n)) == 0
        return n.value
    assert balance(0, 128, 0) % 256 == 0
    assert balance(1000, 128, 0) <= balance(100000, 128, 0)
    assert balance(5000, 128, 1) >= 5000 * 128 * 8
    assert emb(0, 1, 1) % 256 == 0
    assert emb(1, 1, 1) <= emb(1000, 1, 1) <= emb(100000, 1, 1)
    assert emb(1000, 100, 64) <= emb(1000, 100, 4096)
    assert emb(5000, 100, 64) < emb(5000, 100, 4096)
    assert lib.ap_route_balance_scratch_bytes(10, 8, 0, None) == -1
    assert lib.ap_route_balance_scratch_bytes(10, 0, 0, ctypes.byref(n)) == -1
    assert lib.ap_embed_scratch_bytes(10, 8, 0, ctypes.byref(n)) == -1
    assert lib.ap_embed_scratch_bytes(10, 8, 4, None) == -1


def test_binding_refuses_what_it_cannot_pass():
    import torch

    import activation_paging_gb300 as ap
    x = torch.zeros(4, 8)
    for call in (lambda: ap.route_balance(x, 2), lambda: ap.route_backward(x), lambda: ap.embed(x, torch.zeros(3).long()),
                 lambda: ap.embed_backward(x, torch.zeros(4).long(), 10)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


def test_embed_refuses_rows_beyond_its_columns(lib):
    n, H = ctypes.c_int64(0), 2 ** 28 + 1
    assert lib.ap_embed(None, 2, H, 0, None, 4, 1, H, 1.0, None, H, 0, None, None) == -1
    assert b"sizes" in lib.ap_last_error()
    assert lib.ap_embed_scratch_bytes(10, 2, H, ctypes.byref(n)) == -1
    assert lib.ap_embed_scratch_bytes(10, 2, H - 1, ctypes.byref(n)) == 0
