"""GPU parity over every form of routing with its balance loss and of the
router's gradient: each step of the ladder by experts, as one cluster and as two
launches, vectors and single loads, masked and short last groups, ties.

Bounds, all sums being of terms that are not negative (u = 2^-24, p_rel the
relative error of a softmax value):
* prob: a warp adds at most S / W + 1 rows (W warps of a block, 8 or 16), a
  block its W warps, the second kernel at most 3 rows a thread and a tree of 2
  and 5 levels (the cluster: 8 blocks), then one division:
  p_rel + (S / 8 + 1 + 16 + 3 + 7 + 1) u;
* slope: ten roundings;
* loss: of a column's slope (10 u), its sum (as prob) and one product, then the
  columns: E / 256 + 1 a thread, 5 levels, 16 warps, the groups of a block, 8
  blocks in the cluster; 8 columns, G E / 8192 + 1 a thread, 5 levels and 32
  warps in the second kernel.
"""
import numpy as np
import pytest
import torch

from activation_paging_gb300 import inputs
from gpu_util import host, route_tolerance, to_dev
from oracle import training
from test_gpu_balance import U, grad_bound, p_rel

pytestmark = pytest.mark.gpu

ap = pytest.importorskip("activation_paging_gb300")

EXPERTS = [8, 32, 33, 64, 65, 128, 130, 255, 256, 257, 260, 511, 512, 1000, 1023, 1024]
CLUSTER, TWO_LAUNCHES = 200, 1300  # tokens: at most 1024 of at most 2^18 logits in one cluster, else two launches


def case(T, E, k, S, pad, ties=False):
    logits = inputs.router_logits(7 * T + E, T, E, 1.0, 0.4)
    if ties:
        logits = (np.round(logits * 2) / 2).astype(np.float32)
    mask = None
    if pad:
        S1, G = training._groups(T, S)
        length = inputs.rng(T + E, 7).integers(0, S1 + 1, G)
        if G > 2:
            length[1] = 0  # a group whose mask leaves nothing
        mask = ((np.arange(T) % S1) < length[np.arange(T) // S1]).astype(np.uint8)
    return logits, mask


def placed(a, shift):
    """The array on the GPU, `shift` elements into a buffer."""
    buf = torch.empty(a.size + shift, dtype=torch.float32, device="cuda")
    t = buf[shift:].view(a.shape)
    t.copy_(to_dev(a))
    return t


def check(T, E, k, S, pad, shift=0, ties=False):
    logits, mask = case(T, E, k, S, pad, ties)
    m = None if mask is None else to_dev(mask)
    x = placed(logits, shift)
    assert x.data_ptr() % 16 == 4 * shift % 16
    assert (ap.route_balance_scratch_bytes(T, E, S) == 0) == (T <= 1024 and T * E <= 2 ** 18)
    r = ap.route_balance(x, k, coef=0.3, group_tokens=S, mask=m)
    e = training.route_balance(logits, k, 0.3, S, mask)
    S1, G = training._groups(T, S)
    assert np.array_equal(host(r["idx"]), e["idx"]) and np.array_equal(host(r["counts"]), e["counts"])
    assert np.all(np.abs(host(r["w"]) - e["w"]) <= route_tolerance(logits, e["idx"], e["w"]) + U * e["w"])
    prel = float(p_rel(logits).max()) + (S1 / 8 + 28) * U
    assert np.all(np.abs(host(r["prob"]) - e["prob"]) <= prel * e["prob"] + 2.0 ** -120)
    assert np.all(np.abs(host(r["slope"]) - e["slope"]) <= 10 * U * e["slope"])
    terms = 11 + E / 256 + 1 + 5 + 16 + G + 8 + G * E / 8192 + 1 + 5 + 32 + 8
    assert abs(float(r["loss"]) - e["loss"]) <= (prel + terms * U) * e["loss"]
    idx, w = ap.route_topk(x, k)
    assert torch.equal(r["idx"], idx) and torch.equal(r["w"], w)
    # and back
    dw = inputs.rng(T, 11).standard_normal((T, k)).astype(np.float32) * np.float32(0.1)
    wf, sl = e["w"].astype(np.float32), e["slope"].astype(np.float32)
    got = ap.route_backward(x, to_dev(e["idx"]), to_dev(wf), to_dev(dw), to_dev(sl), group_tokens=S, mask=m)
    exp = training.route_backward(logits, e["idx"], wf, dw, sl, 1.0, S, mask)
    assert np.all(np.abs(host(got) - exp) <= grad_bound(logits, e["idx"], wf, dw, sl, 1.0, S1, mask))


@pytest.mark.parametrize("T", [CLUSTER, TWO_LAUNCHES])
@pytest.mark.parametrize("E", EXPERTS)
def test_steps_of_the_ladder(T, E):
    check(T, E, min(E, 8), 0, False)
    check(T, E, min(E, 32), T // 3 + 1, True)       # a short last group
    check(T, E, 1, 7, True)                         # more groups than a cluster has blocks


@pytest.mark.parametrize("T", [CLUSTER, TWO_LAUNCHES])
@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("E", [32, 64, 128, 256, 512, 1024])
def test_logits_off_their_16_byte_boundary(T, E, shift):
    check(T, E, 6, T // 2 + 1, True, shift)


@pytest.mark.parametrize("T", [CLUSTER, TWO_LAUNCHES])
@pytest.mark.parametrize("E", [33, 128, 130, 256, 512, 1023])
def test_many_equal_logits(T, E):
    """More candidates than lanes, and equal ones among them: the lowest ids are chosen."""
    check(T, E, 8, 0, False, ties=True)
    check(T, E, 32, 50, True, ties=True)


@pytest.mark.parametrize("T,E", [(1024, 256), (1025, 256), (1024, 257), (256, 1024), (257, 1024), (5000, 8), (40000, 16)])
def test_sizes_where_the_form_changes(T, E):
    check(T, E, min(8, E), 0, True)
    check(T, E, min(8, E), 333, False)


def test_more_groups_than_blocks_and_more_than_a_block_finishes():
    check(3000, 64, 4, 1, True)      # a group per token
    check(20000, 260, 8, 13, False)  # 1539 groups of 33 pieces
