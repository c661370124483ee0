"""Host logic of a layer's operators (no GPU is touched)."""
import pytest
import torch

from activation_paging_gb300 import AdamW


def test_an_optimizer_knows_where_its_tensors_were():
    """The addresses of what a step writes and reads, and their memory, are held from the start."""
    o = object.__new__(AdamW)
    o.params, o.master = [torch.zeros(3), torch.zeros(0)], None
    o.state, o._names = {"m": torch.zeros(256), "v": torch.zeros(256), "step": torch.zeros(2, dtype=torch.int32)}, ["m", "v", "step"]
    o.grads = [torch.zeros(3), torch.zeros(0)]
    o._held, o._grads_held = o._hold(o._written()), o._hold(o.grads)
    o._stay_written()
    o._stay_grads()
    old = o.params[0].data_ptr()
    o.params[0].data = torch.ones(3)
    assert o.params[0].data_ptr() != old and old in [s.data_ptr() for s in o._held[2]]  # nobody else can have it
    o._stay_grads()
    with pytest.raises(ValueError, match="copy into them"):
        o._stay_written()
    o.params.pop()
    with pytest.raises(ValueError, match="copy into them"):
        o._stay_written()
    o.grads[0] = torch.ones(3)
    with pytest.raises(ValueError, match="bind"):
        o._stay_grads()
