"""The sources of routing by scores, the experts' products and the weights' update:
inputs that the kernel ahead may still write are not promised to stand still, and
waits inside kernels have a limit."""
import os
import re

import pytest

from test_kernels_wait_first import CSRC, KERNELS

FILES = ("scored.cu", "adamw.cu", "experts.cu")


@pytest.mark.parametrize("file,name,params,body", [k for k in KERNELS if k[0] in FILES], ids=[k[1] for k in KERNELS if k[0] in FILES])
def test_inputs_are_not_promised_to_stand_still(file, name, params, body):
    assert not re.findall(r"const\s+\w+\s*\*\s*__restrict__\s+(\w+)", params)


def test_every_file_has_kernels():
    assert {k[0] for k in KERNELS if k[0] in FILES} == set(FILES)


def test_waits_have_a_limit():
    """mbarrier waits stand in one place only, inside a counted loop."""
    for file in ("experts.cu", "umma.cuh"):
        with open(os.path.join(CSRC, file)) as f:
            text = f.read()
        assert text.count("mbarrier.try_wait") == (1 if file == "umma.cuh" else 0)
        assert "mbarrier.test_wait" not in text and not re.search(r"while\s*\(\s*(true|1)\s*\)|for\s*\(\s*;\s*;\s*\)", text)
    with open(os.path.join(CSRC, "umma.cuh")) as f:
        wait = re.search(r"bool bar_wait\(.*?\n}", f.read(), flags=re.S).group(0)
    assert re.search(r"for \(uint32_t i = 0; i < kTries; \+\+i\)", wait)
