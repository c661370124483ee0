"""GPU: the table's gradient written whole, call after call with other ids over
one work space and one table, where the kernels of a call overlap and the work
space holds what the call before left in it.

Each id set's first result is held against its 64-bit form, with the bound of a
sum of n rows in single precision ((n + 2) 2^-24 of the sum of magnitudes) and
one rounding to the table's type (2^-8 relative for BF16); every later result has
to equal the first bit for bit.  The table is filled with a value before each
call, so that a row which is not written shows."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ap = pytest.importorskip("activation_paging_gb300")

U = 2.0 ** -24
SETS = 5


def zipf_ids(g, T, V):
    cdf = torch.cumsum(1.0 / torch.arange(1, V + 1, device="cuda", dtype=torch.float64), 0)
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64) * cdf[-1]
    return torch.searchsorted(cdf, u).clamp_(max=V - 1)


def id_sets(T, V, seed):
    """Zipf ids as text has them, the same turned round (other rows named), uniform ids, one id, and a third padding."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    sets = [zipf_ids(g, T, V), V - 1 - zipf_ids(g, T, V), torch.randint(0, V, (T,), generator=g, device="cuda"),
            torch.full((T,), V // 3, device="cuda"), zipf_ids(g, T, V)]
    sets[4][::3] = V - 1
    assert len(sets) == SETS
    return sets


def check_exact(got, dout, ids, V, pad, scale):
    keep = torch.nonzero(ids != pad).flatten()
    names, inv = torch.unique(ids[keep], return_inverse=True)
    rows = dout[keep].double()
    total = torch.zeros(len(names), dout.shape[1], dtype=torch.float64, device="cuda").index_add_(0, inv, rows)
    size = torch.zeros_like(total).index_add_(0, inv, rows.abs()).mul_(abs(scale))
    n = torch.bincount(inv, minlength=len(names)).double()[:, None]
    total *= scale
    bound = size * (n + 2) * U
    if got.dtype == torch.bfloat16:
        bound += (total.abs() + bound) * 2.0 ** -8 + 2.0 ** -130
    else:
        bound += total.abs() * U
    off = (got[names].double() - total).abs() - bound
    assert float(off.max()) <= 0, (int((off > 0).any(1).sum()), "rows off")
    unnamed = torch.ones(V, dtype=torch.bool, device="cuda")
    unnamed[names] = False
    assert not bool((got != 0).any(1)[unnamed].any())


def same(a, b):
    """Bit for bit, and where not: how many rows differ."""
    if torch.equal(a, b):
        return True
    pytest.fail("%d rows differ" % int((a != b).any(1).sum()))


SHAPES = [  # T, V, H, types of rows and table, calls of the eager and of the graph run
    (16384, 151936, 2048, torch.bfloat16, torch.bfloat16, 200, 40),
    (3000, 151936, 2048, torch.bfloat16, torch.bfloat16, 200, 40),
    (8192, 131072, 1024, torch.bfloat16, torch.float32, 100, 20),
    (16385, 151936, 515, torch.float32, torch.bfloat16, 100, 20),   # rows off 16-byte boundaries
    (140000, 151936, 512, torch.bfloat16, torch.bfloat16, 100, 20),  # longer than one cluster sorts
]


@pytest.mark.parametrize("T,V,H,rows,table,calls,replays", SHAPES)
def test_whole_gradients_in_turn_over_one_work_space(T, V, H, rows, table, calls, replays):
    g = torch.Generator(device="cuda").manual_seed(T + H)
    pad, scale = V - 1, 1.5
    sets = id_sets(T, V, T)
    dout = torch.empty(T, H, dtype=rows, device="cuda").normal_(0, 1, generator=g)
    out = torch.empty(V, H, dtype=table, device="cuda")
    scratch = torch.full((ap.embed_scratch_bytes(T, V, H),), 0xA5, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(ids):
        ap.embed_backward(dout, ids, V, scale=scale, padding_idx=pad, dtable=out, scratch=scratch, status=status)
    first = []
    for ids in sets:
        out.fill_(7.0)
        call(ids)
        check_exact(out, dout, ids, V, pad, scale)
        first.append(out.clone())
    order = np.random.default_rng(T).integers(0, SETS, calls)
    for q in order:  # eager, each call checked
        out.fill_(7.0)
        call(sets[q])
        assert same(out, first[q])
    for q in range(calls):  # calls back to back, the last one checked
        for r in range(3):
            call(sets[(q + r) % SETS])
        assert same(out, first[(q + 2) % SETS])
    graph, ids = torch.cuda.CUDAGraph(), sets[0].clone()
    with torch.cuda.graph(graph):
        out.fill_(7.0)
        call(ids)
    for q in range(replays):
        ids.copy_(sets[q % SETS])
        graph.replay()
        assert same(out, first[q % SETS])
    torch.cuda.synchronize()
    assert int(status) == 0


def test_whole_gradients_of_several_tables_in_turn():
    """As a step with several tables calls it: each call allocates its work space, which the one before freed."""
    T, V, H = 16384, 151936, 1024
    g = torch.Generator(device="cuda").manual_seed(3)
    sets = id_sets(T, V, 9)
    douts = [torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g) for _ in sets]
    first = []
    for ids, d in zip(sets, douts):
        first.append(ap.embed_backward(d, ids, V, padding_idx=V - 1, dtype=torch.bfloat16))
        check_exact(first[-1], d, ids, V, V - 1, 1.0)
    tables = [torch.full_like(t, 7.0) for t in first]
    for _ in range(60):
        for t in tables:
            t.fill_(7.0)
        for ids, d, t in zip(sets, douts, tables):
            ap.embed_backward(d, ids, V, padding_idx=V - 1, dtable=t)
        for t, e in zip(tables, first):
            assert same(t, e)
