"""Host logic of a layer's operators (no GPU is touched)."""
import ctypes

import numpy as np
import pytest
import torch

from activation_paging_gb300 import AdamW, _lib, build
from activation_paging_gb300._lib import AdamWConfig, AdamWTensor
from oracle import layer


def build_lib():
    build.build()
    return _lib.load()


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


def test_refused_roundings():
    with pytest.raises(ValueError, match="rounding"):
        AdamW([torch.zeros(3)], [torch.zeros(3)], rounding="nearest")
    lib = build_lib()
    t = (AdamWTensor * 1)()
    c = AdamWConfig(beta1=0.9, beta2=0.99, param_dtype=2, grad_dtype=2, state_bits=8, rounding=2, d_step=4096)
    n0 = lib.ap_launch_count()
    assert lib.ap_adamw_step(t, 1, ctypes.byref(c), None) == -1 and b"rounding" in lib.ap_last_error()
    assert lib.ap_launch_count() == n0


def test_codes_rounded_by_values_are_fair_to_them():
    """All 65536 fractions once: the mean of the decoded values is the value, to half of 2^-16 of a step; the codes' own
    rounding is a quarter of a scale too large at a fraction of one half."""
    r = np.arange(65536) / 65536.0
    for x in (0.0, 0.16, 0.25, 1.0, 1.6, 2.25, 6.5, 65.3, 8000.7):
        for power in (1, 2):
            c = layer.adamw_codes(np.full(65536, x), r, 255, power, "values")
            step = (np.floor(np.sqrt(x)) + 1) ** (2 * power) - np.floor(np.sqrt(x)) ** (2 * power)
            assert abs((c ** (2 * power)).mean() - x ** power) <= step * 2.0 ** -17 * 1.001
    c = layer.adamw_codes(np.full(65536, 2.25), r, 255, 1)
    assert abs((c * c).mean() - 2.5) < 1e-9
