"""GPU: the training operators on streams of SM partitions (green contexts),
which take smaller clusters of thread blocks than the whole GPU: the results
have the bits that they have on an ordinary stream."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

ap = pytest.importorskip("activation_paging_gb300")


@pytest.fixture(params=[8, 24, 100])
def partition(request):
    """Streams of two disjoint partitions, of at least so many SMs and of the others."""
    from activation_paging_gb300 import build as cuda_build
    lib = ctypes.CDLL(cuda_build.BENCH_LIB)
    vp, ip = ctypes.c_void_p, ctypes.c_int
    lib.apb_green_split.restype = ip
    lib.apb_green_split.argtypes = [ip, ip] + [ctypes.POINTER(vp)] * 2 + [ctypes.POINTER(ip)] * 2 + \
        [ctypes.POINTER(vp)] * 2
    lib.apb_green_destroy.restype = ip
    lib.apb_green_destroy.argtypes = [vp] * 4
    s1, s2, c1, c2 = vp(), vp(), vp(), vp()
    n1, n2 = ip(), ip()
    rc = lib.apb_green_split(torch.cuda.current_device(), request.param, ctypes.byref(s1), ctypes.byref(s2),
                             ctypes.byref(n1), ctypes.byref(n2), ctypes.byref(c1), ctypes.byref(c2))
    if rc < 0:
        pytest.skip(f"the driver lacks green-context entry point {-rc} of apb_green_split")
    assert rc == 0, f"green context split failed: CUDA driver error {rc}"
    yield torch.cuda.ExternalStream(s1.value), torch.cuda.ExternalStream(s2.value)
    torch.cuda.synchronize()
    assert lib.apb_green_destroy(s1, s2, c1, c2) == 0


def on(stream, call):
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        r = call()
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    return r


@pytest.mark.parametrize("T", [900, 1500, 8192, 8193, 20000, 65536, 65537, 140000])
def test_embedding_gradient_on_partitions(partition, T):
    """Sorts of one block, of clusters of 8 where 16 do not fit, and over memory where the tokens are too many for that."""
    V, H = 4000, 72
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = (torch.rand(T, generator=g, device="cuda") ** 3 * V).long()
    dout = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    old = torch.randn(V, H, generator=g, device="cuda")
    whole = ap.embed_backward(dout, ids, V, padding_idx=7)
    added = ap.embed_backward(dout, ids, V, dtable=old.clone(), accumulate=True)
    for s in partition:
        assert torch.equal(on(s, lambda: ap.embed_backward(dout, ids, V, padding_idx=7)), whole)
        kept = old.clone()
        assert torch.equal(on(s, lambda: ap.embed_backward(dout, ids, V, dtable=kept, accumulate=True)), added)


@pytest.mark.parametrize("T,E,k,S", [(40, 8, 2, 0), (300, 64, 6, 100), (1000, 128, 8, 0), (256, 1000, 8, 1), (6000, 96, 4, 512)])
def test_balance_and_router_gradient_on_partitions(partition, T, E, k, S):
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn(T, E, generator=g, device="cuda")
    a = ap.route_balance(logits, k, coef=0.1, group_tokens=S)
    d = ap.route_backward(logits, a["idx"], a["w"], a["w"], a["slope"], group_tokens=S)
    for s in partition:
        b = on(s, lambda: ap.route_balance(logits, k, coef=0.1, group_tokens=S))
        for n in ("idx", "w", "counts", "prob", "slope", "loss"):
            assert torch.equal(a[n], b[n]), n
        assert torch.equal(on(s, lambda: ap.route_backward(logits, b["idx"], b["w"], b["w"], b["slope"], group_tokens=S)), d)
