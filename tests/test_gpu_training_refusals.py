"""GPU: the bindings of the training operators refuse tensors that the kernels
could not write to: work space off the GPU, status words off the GPU, too short
or between two words."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ap = pytest.importorskip("activation_paging_gb300")


def calls(status):
    logits, ids = torch.zeros(4, 8, device="cuda"), torch.tensor([0, 1, 2, 9], device="cuda")
    r = ap.route_balance(logits, 2)
    bad = torch.full_like(r["idx"], 99)
    return (lambda: ap.route_backward(logits, bad, r["w"], r["w"], r["slope"], status=status),
            lambda: ap.embed(logits, ids, status=status), lambda: ap.embed_backward(logits, ids, 5, status=status))


@pytest.mark.parametrize("kind", ["cpu", "short", "empty", "unaligned"])
def test_status_words(kind):
    status = {"cpu": lambda: torch.zeros(1, dtype=torch.int32),
              "short": lambda: torch.zeros(3, dtype=torch.uint8, device="cuda"),
              "empty": lambda: torch.zeros(0, dtype=torch.int32, device="cuda"),
              "unaligned": lambda: torch.zeros(9, dtype=torch.uint8, device="cuda")[1:]}[kind]()
    for call in calls(status):
        with pytest.raises(ValueError, match="status"):
            call()


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64, torch.uint8])
def test_status_words_of_any_type(dtype):
    for q in range(3):
        status = torch.zeros(8, dtype=dtype, device="cuda")
        calls(status)[q]()
        assert int(status[0]) == ap.FLAG_BAD_INDEX


def test_work_space_of_routing():
    T, E = 5000, 16
    logits = torch.zeros(T, E, device="cuda")
    n = ap.route_balance_scratch_bytes(T, E)
    for bad in (torch.empty(n, dtype=torch.uint8), torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="scratch"):
            ap.route_balance(logits, 2, out={"scratch": bad})
    for dtype in (torch.uint8, torch.float32):
        kept = torch.empty(n, dtype=dtype, device="cuda")
        assert ap.route_balance(logits, 2, out={"scratch": kept})["scratch"] is kept


def test_gradient_of_the_weights_has_two_dimensions():
    logits = torch.zeros(4, 8, device="cuda")
    r = ap.route_balance(logits, 1)
    with pytest.raises(ValueError, match="dw"):
        ap.route_backward(logits, r["idx"], r["w"], r["w"][:, 0])
