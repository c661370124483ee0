"""GPU parity: the embedding lookup and its gradient against their 64-bit plain
forms.

The lookup makes one single-precision product and one rounding to the output's
type, so it is compared bit for bit with the same two roundings on the host.
The gradient of an id with n tokens is a sum of n rows in single precision
(n - 1 additions in any order: relative (n + 2) 2^-24 of the sum of
magnitudes), a product, an addition to the kept gradient, and one rounding to
the table's type (half a unit in the last place: 2^-8 relative for BF16, whose values
have 8 significant bits)."""
import numpy as np
import pytest
import torch

from activation_paging_gb300 import inputs
from gpu_util import bf16_to_dev, bf16_to_host, host, to_dev
from oracle import training

pytestmark = pytest.mark.gpu

ap = pytest.importorskip("activation_paging_gb300")

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rows(seed, n, H, dtype, extra=0, shift=0):
    """(device rows, float64 values): n rows of H values, `extra` elements between rows, the first `shift` elements
    into a buffer."""
    a = inputs.rng(seed, 21).standard_normal((n, H)).astype(np.float32)
    if dtype == "bf16":
        a = inputs.bf16_bits_to_f32(inputs.f32_to_bf16_bits(a))
    buf = torch.full((shift + n * (H + extra) + H,), 7.0, dtype=DT[dtype], device="cuda")
    t = buf[shift:shift + n * (H + extra)].view(n, H + extra)[:, :H]
    t.copy_(to_dev(a))
    return t, a.astype(np.float64), buf


def f32_of(t):
    return host(t.float())


def zipf_ids(seed, T, V):
    g = inputs.rng(seed, 22)
    p = 1.0 / np.arange(1, V + 1)
    return g.choice(V, T, p=p / p.sum())


SHAPES = [  # T, V, H, extra elements between rows, shift of the first row
    (1, 1, 1, 0, 0),
    (1, 50, 2048, 0, 0),
    (3, 7, 8, 0, 0),
    (33, 1000, 1001, 0, 0),     # odd rows
    (64, 300, 130, 2, 0),
    (100, 300, 256, 8, 0),      # rows apart
    (257, 4099, 512, 0, 1),     # rows off their 16-byte boundary
    (500, 97, 72, 0, 0),
    (1000, 32003, 264, 0, 0),
]


@pytest.mark.parametrize("table,out", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("T,V,H,extra,shift", SHAPES)
def test_embed_matches_plain_form(T, V, H, extra, shift, table, out):
    tab, a, _ = rows(T, V, H, table, extra, shift)
    o, _, buf = rows(T + 1, T, H, out, extra, shift)
    ids = zipf_ids(T, T, V)
    scale = np.float32(0.37)
    got = ap.embed(tab, to_dev(ids.astype(np.int64 if T % 2 else np.int32)), scale=float(scale), out=o)
    exp = a.astype(np.float32)[ids] * scale
    if out == "bf16":
        assert np.array_equal(bf16_to_host(got), inputs.f32_to_bf16_bits(exp))
    else:
        assert np.array_equal(host(got), exp)
    exact = training.embed(a, ids, float(scale))
    assert np.all(np.abs(f32_of(got) - exact) <= (2.0 ** -8 if out == "bf16" else 2 * U) * np.abs(exact))
    # nothing between the rows, before or after them was written
    rest = buf.clone()
    rest[shift:shift + T * (H + extra)].view(T, H + extra)[:, :H] = 7.0
    assert bool((rest == 7.0).all())


@pytest.mark.parametrize("extra,to_extra", [(0, 0), (1, 0), (0, 1), (3, 4)])
@pytest.mark.parametrize("shift,to_shift", [(0, 0), (1, 0), (0, 1), (1, 1), (5, 2)])
@pytest.mark.parametrize("H", [1, 2, 3, 15, 64, 65, 511, 513, 1025])
def test_embed_bf16_rows_that_start_between_pairs(H, shift, to_shift, extra, to_extra):
    """Each row of the table to rows of either parity, its first and last row and bad ids among them."""
    V = 7
    ids = np.array([0, 0, V - 1, V - 1, 1, 1, V - 2, V - 2, -1, V, 3, 4, 5, 0, V - 1], np.int64)
    tab, a, _ = rows(H, V, H, "bf16", extra, shift)
    o, _, buf = rows(H + 1, len(ids), H, "bf16", to_extra, to_shift)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = bf16_to_host(ap.embed(tab, to_dev(ids), scale=0.37, out=o, status=status))
    good = (ids >= 0) & (ids < V)
    exp = a.astype(np.float32)[np.where(good, ids, 0)] * np.float32(0.37) * good[:, None]
    assert np.array_equal(got[good], inputs.f32_to_bf16_bits(exp)[good]) and not got[~good].any()
    assert int(host(status)[0]) == ap.FLAG_BAD_INDEX
    rest = buf.clone()
    pitch = H + to_extra
    rest[to_shift:to_shift + len(ids) * pitch].view(len(ids), pitch)[:, :H] = 7.0
    assert bool((rest == 7.0).all())


def test_embed_ids_outside_are_zero_rows_and_flagged():
    tab, a, _ = rows(1, 10, 24, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = torch.tensor([3, -1, 10, 2 ** 40, -2 ** 40, 9], device="cuda")
    got = f32_of(ap.embed(tab, ids, status=status))
    assert int(host(status)[0]) == ap.FLAG_BAD_INDEX
    assert np.array_equal(got[[0, 5]], a[[3, 9]]) and not got[1:5].any()
    status.zero_()
    ap.embed(tab, ids[:1], status=status)
    assert int(host(status)[0]) == 0
    assert ap.embed(tab, ids[:0]).shape == (0, 24)


def test_embed_passes_infinities_and_nan_on():
    tab = torch.zeros(3, 16, device="cuda")
    tab[1, 2], tab[1, 3], tab[2, 5] = float("inf"), float("-inf"), float("nan")
    got = host(ap.embed(tab, torch.tensor([0, 1, 2], device="cuda"), scale=2.0, dtype=torch.bfloat16).float())
    assert got[1, 2] == np.inf and got[1, 3] == -np.inf and np.isnan(got[2, 5])
    assert np.isfinite(got[0]).all() and np.isfinite(np.delete(got[2], 5)).all()


def check_backward(ids, V, H, dout="bf16", grad="f32", accumulate=True, pad=None, extra=0, shift=0, scale=1.5, seed=0,
                   wide=True):
    T = len(ids)
    d, a, _ = rows(seed + 5, T, H, dout, extra, shift)
    g, old, buf = rows(seed + 6, V, H, grad, extra, shift)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ap.embed_backward(d, to_dev(np.asarray(ids, np.int64 if wide else np.int32)), V, scale=scale, padding_idx=pad,
                            dtable=g, accumulate=accumulate, status=status)
    exp, n, size = training.embed_backward(a, ids, V, scale, -1 if pad is None else pad, old if accumulate else None)
    res = f32_of(got).astype(np.float64)
    bound = size * (n[:, None] + 2) * U + np.abs(old) * (U if accumulate else 0)
    if grad == "bf16":
        bound += (np.abs(exp) + bound) * 2.0 ** -8 + 2.0 ** -130
    err = np.abs(res - exp)
    assert np.all(err <= bound + np.abs(exp) * U), (err - bound).max()
    untouched = n == 0
    assert np.array_equal(res[untouched], old[untouched] if accumulate else np.zeros_like(old[untouched]))
    rest = buf.clone()
    rest[shift:shift + V * (H + extra)].view(V, H + extra)[:, :H] = 7.0
    assert bool((rest == 7.0).all())
    bad = [i for i in ids if (i < 0 or i >= V) and i != pad]
    assert int(host(status)[0]) == (ap.FLAG_BAD_INDEX if bad else 0)
    return got


@pytest.mark.parametrize("dout,grad", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("T,V,H,extra,shift", SHAPES)
def test_embed_backward_matches_plain_form(T, V, H, extra, shift, dout, grad, accumulate):
    check_backward(zipf_ids(T, T, V), V, H, dout, grad, accumulate, None, extra, shift, wide=T % 2 == 1)


@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("T", [1, 31, 32, 33, 64, 65, 1000, 2047, 2048, 2049, 5000])
def test_one_id_takes_every_token(T, accumulate):
    check_backward(np.full(T, 5), 11, 40, accumulate=accumulate)


@pytest.mark.parametrize("lengths", [[32, 32, 32], [31, 1, 33, 63, 64, 65], [1] * 200, [500, 1, 700, 2, 3000],
                                     [16, 48, 16, 48, 97]])
def test_runs_that_end_at_and_cross_tiles(lengths):
    ids = np.repeat(np.arange(len(lengths)) * 3 + 1, lengths)
    inputs.rng(len(ids), 23).shuffle(ids)
    for accumulate in (True, False):
        check_backward(ids, 3 * len(lengths) + 4, 72, accumulate=accumulate)
        check_backward(ids, 3 * len(lengths) + 4, 37, "f32", "f32", accumulate)


@pytest.mark.parametrize("dout,grad", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("H,extra,shift", [(1, 0, 0), (3, 0, 1), (37, 0, 0), (130, 2, 0), (257, 0, 1), (264, 0, 2),
                                           (514, 0, 0), (1001, 3, 0), (2056, 0, 0)])
def test_many_tokens_with_rows_that_start_anywhere(H, extra, shift, dout, grad):
    """Long enough for the staged sums: rows on and off 16-byte boundaries, buffers that begin and end inside one."""
    ids = zipf_ids(H, 3000, 700)
    ids[::7] = 699
    for accumulate in (True, False):
        check_backward(ids, 700, H, dout, grad, accumulate, 5, extra, shift)


@pytest.mark.parametrize("accumulate", [True, False])
def test_padding_and_bad_ids(accumulate):
    T, V = 700, 60
    ids = zipf_ids(9, T, V).astype(np.int64)
    ids[500:] = 0
    check_backward(ids, V, 64, accumulate=accumulate, pad=0)
    check_backward(ids, V, 64, accumulate=accumulate, pad=V - 1)
    ids[[3, 99, 200]] = [-1, V, 2 ** 33 + 5]
    check_backward(ids, V, 64, accumulate=accumulate)
    check_backward(ids, V, 64, accumulate=accumulate, pad=0)
    check_backward(np.full(300, 4), V, 64, accumulate=accumulate, pad=4)      # only padding
    check_backward(np.full(300, -7), V, 64, accumulate=accumulate)            # only bad ids


@pytest.mark.parametrize("T", [16, 17, 255, 256, 257, 1023, 1024, 1025, 131072, 131073])
def test_lengths_where_the_form_changes(T):
    """One piece of a run or two, ranking by counting or by passes, one launch or three, one cluster or passes over
    memory; a quarter of the tokens share an id, the others are spread."""
    ids = inputs.rng(T, 25).integers(0, 900, T)
    ids[::4] = 901
    check_backward(ids, 902, 12, "bf16", "f32", True)
    check_backward(ids, 902, 12, "f32", "bf16", False, pad=901)


@pytest.mark.parametrize("T", [40, 2000])
def test_an_id_of_minus_one_is_a_bad_one(T):
    ids = zipf_ids(T, T, 50).astype(np.int64)
    ids[7] = -1
    check_backward(ids, 50, 24)          # no padding: flagged
    check_backward(ids, 50, 24, pad=3)


@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("T", [6, 3000])
@pytest.mark.parametrize("H,extra,shift", [(1, 0, 0), (2, 0, 1), (5, 0, 3), (7, 1, 1), (8, 0, 0), (101, 0, 5), (9001, 0, 1)])
def test_zeros_between_named_rows(H, extra, shift, T, grad):
    """A gradient written whole: spans of rows that no id names, from none to many rows, start and end anywhere."""
    check_backward(np.resize([0, 5, 6, 31, 32, 69], T), 70, H, "f32", grad, False, None, extra, shift)
    check_backward(np.resize([1, 3, 68], T), 70, H, "f32", grad, False, None, extra, shift)


@pytest.mark.parametrize("accumulate", [True, False])
def test_no_tokens(accumulate):
    check_backward(np.zeros(0, np.int64), 9, 24, accumulate=accumulate)


@pytest.mark.parametrize("T,V,H", [(3000, 1023, 8), (3000, 1024, 8), (5000, 2 ** 20 - 1, 4), (5000, 2 ** 20 + 3, 4),
                                   (20000, 151936, 16), (70000, 151936, 8), (300000, 40000, 8)])
def test_vocabulary_and_length_ranges(T, V, H):
    """Keys of one to three radix digits, and lengths of every form of the sort."""
    check_backward(zipf_ids(T, T, V), V, H, "f32", "f32", True, pad=3)
    ids = inputs.rng(T, 24).integers(0, V, T)
    check_backward(ids, V, H, "bf16", "f32", False)


def test_offsets_beyond_32_bits():
    """A table and a gradient of more than 2^32 elements (rows far apart): lookups and sums at its end."""
    V, H, pitch = 3, 64, 2200000000
    tab = torch.empty(2 * pitch + H, dtype=torch.bfloat16, device="cuda").as_strided((V, H), (pitch, 1))
    vals = torch.arange(V * H, device="cuda").view(V, H).float() / 16
    tab.copy_(vals)
    ids = torch.tensor([2, 1, 0, 2], device="cuda")
    assert torch.equal(ap.embed(tab, ids, dtype=torch.float32), vals[ids])
    d = torch.ones(4, H, device="cuda")
    ap.embed_backward(d, ids, V, dtable=tab, accumulate=False)
    assert torch.equal(tab.float(), torch.tensor([1.0, 1.0, 2.0], device="cuda")[:, None].expand(V, H))


def test_equal_inputs_give_equal_bits():
    T, V, H = 20000, 5000, 264
    ids = to_dev(zipf_ids(3, T, V))
    d = torch.randn(T, H, device="cuda")
    a = ap.embed_backward(d, ids, V)
    for _ in range(5):
        assert torch.equal(a, ap.embed_backward(d, ids, V))


def test_gradient_matches_differences_of_the_lookup():
    """f(table) = <dout, embed(table)> is linear: the difference for a step of one element is its gradient, up to the
    roundings of the products and of the difference."""
    T, V, H = 40, 7, 12
    ids = to_dev(zipf_ids(4, T, V))
    tab, d = torch.randn(V, H, device="cuda"), torch.randn(T, H, device="cuda")
    g = host(ap.embed_backward(d, ids, V, scale=0.75)).astype(np.float64)

    def f(t):
        return float((ap.embed(t, ids, scale=0.75).double() * d.double()).sum())
    base = f(tab)
    size = float((ap.embed(tab, ids, scale=0.75).abs() * d.abs()).sum() + d.abs().sum())
    for v in range(V):
        for h in range(0, H, 5):
            t = tab.clone()
            t[v, h] += 1.0
            assert abs(f(t) - base - g[v, h]) <= 8 * U * size


def test_scratch_reuse_stream_and_graph():
    T, V, H = 3000, 800, 128
    d = torch.randn(T, H, device="cuda").bfloat16()
    ids = to_dev(zipf_ids(5, T, V))
    a = ap.embed_backward(d, ids, V)
    scratch = torch.full((ap.embed_scratch_bytes(T, V, H),), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(a, ap.embed_backward(d, ids, V, scratch=scratch))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = ap.embed_backward(d, ids, V, stream=s)
    x = ap.embed(b, ids, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, b) and torch.equal(x, a[ids])
    g = torch.cuda.CUDAGraph()
    out = torch.empty(V, H, device="cuda")
    with torch.cuda.graph(g):
        ap.embed_backward(d, ids, V, dtable=out, scratch=scratch)
    ids.copy_(to_dev(zipf_ids(6, T, V)))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ap.embed_backward(d, ids, V))


def test_binding_refuses():
    tab = torch.zeros(4, 8, device="cuda")
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    bad = [
        lambda: ap.embed(tab.half(), ids),
        lambda: ap.embed(tab.t(), ids),
        lambda: ap.embed(tab, ids.short()),
        lambda: ap.embed(tab, ids[:, None]),
        lambda: ap.embed(tab, ids, dtype=torch.float16),
        lambda: ap.embed(tab, ids, out=torch.zeros(2, 8, device="cuda")),
        lambda: ap.embed_backward(tab, ids, 9),                    # four rows, three ids
        lambda: ap.embed_backward(tab[:3], ids, 9, accumulate=True),
        lambda: ap.embed_backward(tab[:3], ids, 9, dtable=torch.zeros(8, 8, device="cuda")),
        lambda: ap.embed_backward(tab[:3].expand(3, 8)[:1].expand(3, 8), ids, 9, dtable=tab[:1].expand(9, 8)),
        lambda: ap.route_balance(tab, 2, mask=torch.ones(3, dtype=torch.bool, device="cuda")),
        lambda: ap.route_balance(tab, 2, mask=torch.ones(4, device="cuda")),
        lambda: ap.route_backward(tab, dw=torch.zeros(4, 2, device="cuda")),
        lambda: ap.route_backward(tab, slope=torch.zeros(2, 8, device="cuda")),
        lambda: ap.route_backward(tab, dloss=torch.zeros(2, device="cuda")),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ap.APError):
        ap.route_balance(tab, 9)
    with pytest.raises(ap.APError):
        ap.embed_backward(tab[:3], ids, 4, padding_idx=4)
