"""GPU parity of the embedding gradient at lengths that reach each form of its
sort: 1, 2, 4 and 8 tokens a thread of one cluster, and passes over memory whose
digit counts are scanned in one turn of the scan's cluster and in several."""
import numpy as np
import pytest

from activation_paging_gb300 import inputs
from test_gpu_embed import check_backward, zipf_ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,H", [
    (16384, 900, 8),      # one token a thread of 16 blocks
    (32768, 151936, 8),   # two
    (40000, 900, 8),      # four
    (65536, 151936, 8),
    (65537, 900, 8),      # eight
    (131072, 151936, 4),
    (131073, 151936, 4),  # over memory: two passes of 9 bits, 33280 counts (one turn takes 131072)
    (300000, 900, 4),     # one pass of 10 bits, 150528 counts: two turns
    (600000, 151936, 4),  # two passes, two turns each
    (900000, 900, 2),     # four turns
])
def test_every_form_of_the_sort(T, V, H):
    ids = inputs.rng(T + V, 25).integers(0, V, T)
    ids[::5] = V // 2
    check_backward(ids, V, H, "bf16", "f32", True)
    check_backward(zipf_ids(T, T, V), V, H, "f32", "bf16", False, pad=1)


@pytest.mark.parametrize("V", [1, 2, 3, 1023, 1024, 2 ** 20 - 1, 2 ** 20])
@pytest.mark.parametrize("T", [1500, 140000])
def test_vocabularies_at_the_ends_of_a_digit(T, V):
    ids = np.where(inputs.rng(T, 26).random(T) < 0.1, V - 1, inputs.rng(V, 27).integers(0, V, T))
    check_backward(ids, V, 3, "f32", "f32", False)
    check_backward(ids, V, 3, "bf16", "f32", True, pad=V - 1)
