"""Host logic of a layer's operators (no GPU is touched)."""
import ctypes
import os
import re

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


CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "activation_paging_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", " ", f.read(), flags=re.S)


def test_waits_for_whole_sections_go_by_progress():
    """A wait gives up after 2^20 tries, ten milliseconds at the least.  The writers' wait is for all stages of a section, of
    0.34 us and more each: of one expert's 2^31 rows, 11 s.  So it has to start anew as stages are fetched; what is left behind
    the last one fetched is the ring, and no other wait is for more than the ring and an epilogue."""
    text, least_s, stage_s = source("experts.cu"), 0.01, 0.43e-6
    assert (2 ** 31 // 64) * 0.34e-6 > least_s
    wait = re.search(r"bool bar_wait\(.*?\n}", source("umma.cuh"), flags=re.S).group(0)
    assert re.search(r"if \(moved && \*moved != seen\) \{\s*seen = \*moved;\s*i = 0;", wait)
    assert "kTries = 1u << 20" in source("umma.cuh")
    waits = re.findall(r"bar_wait\(((?:[^()]|\([^()]*\))*)\)", text)
    done = [w for w in waits if "s_done" in w]
    assert done and all(w.rstrip().endswith("dead, fetched") for w in done)
    assert re.search(r"fetch<OP, PAIR>\([^;]*;\s*\*\(volatile uint32_t \*\)&s_fetched = \+\+count;", text)
    ring = int(re.search(r"kMaxStages = (\d+)", text).group(1))
    assert 1000 * ring * stage_s < least_s


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_plain_gradient_leaves_out_pairs_that_do_not_count(score, renorm):
    """Against torch's own, of weights that are 0 for such pairs."""
    g = np.random.default_rng(1)
    logits = g.standard_normal((30, 8)).astype(np.float32)
    logits[g.random((30, 8)) < 0.4] = -np.inf
    logits[:, 2] = 0.5
    idx, w, _, eligible = layer.route_scored(logits, 4, score, None, 4, 2, 2, renorm, 1.5)
    assert not eligible.all() and not w[~eligible].any()
    dw = g.standard_normal((30, 4))
    x = torch.tensor(logits, dtype=torch.float64, requires_grad=True)
    s = (torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)).gather(1, torch.from_numpy(idx).long())
    s = torch.where(torch.from_numpy(eligible), s, torch.zeros((), dtype=torch.float64))
    v = 1.5 * (s / s.sum(1, keepdim=True) if renorm else s)
    np.testing.assert_allclose(v.detach().numpy(), w, rtol=1e-6)
    (v * torch.from_numpy(dw)).sum().backward()
    got = layer.route_scored_backward(logits, idx, dw, score, renorm, 1.5, eligible)
    np.testing.assert_allclose(got, np.nan_to_num(x.grad.numpy()), rtol=1e-9, atol=1e-13)
