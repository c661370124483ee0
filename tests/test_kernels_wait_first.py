"""Every kernel of the library is launched so that it may start while the kernel
before it still runs.  Only its own wait (in pdl_begin or pdl_begin_after) makes
what earlier kernels wrote visible to it, and only after it may it write what
they still read.  So the sources are read here: nothing stands before a kernel's
wait but the arrival at its cluster's first barrier, and prefetches, which
change no result."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "activation_paging_gb300", "csrc")
HEAD = re.compile(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\(")
MAY_STAND_BEFORE = re.compile(r"(?:cluster_arrive\(\);|prefetch_inputs<[^;{}]*>\([^;{}]*\);"
                              r"|\{\s*const int64_t t0 = [^;{}]*;\s*prefetch_rows_l2\([^;{}]*\);\s*\}|\s)*")


def _closed(text, at, pair):
    """The end of the bracket that opens at text[at]."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if not depth:
            return i
    raise AssertionError("unbalanced " + pair)


def kernels():
    """(file, name, parameters, body) of every kernel of the library, without comments."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*|/\*.*?\*/", " ", f.read(), flags=re.S)
        for m in HEAD.finditer(text):
            end = _closed(text, m.end() - 1, "()")
            rest = text[end + 1:].lstrip()
            if rest.startswith("{"):
                start = text.index("{", end)
                found.append((os.path.basename(path), m.group(1), text[m.end():end], text[start + 1:_closed(text, start, "{}")]))
    return found


KERNELS = kernels()


def test_all_kernels_are_found():
    names = {k[1] for k in KERNELS}
    assert {"k_embed_sum", "k_embed_join", "k_sort_cluster", "k_balance_finish", "k_route_backward"} <= names
    declared = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")):
        with open(path) as f:
            declared += len(re.findall(r"^(?:template[^\n]*\n)?__global__", f.read(), flags=re.M))
    assert len(KERNELS) >= declared > 20


@pytest.mark.parametrize("file,name,params,body", KERNELS, ids=[k[0] + ":" + k[1] for k in KERNELS])
def test_nothing_but_hints_before_the_wait(file, name, params, body):
    at = re.search(r"\bpdl_begin(?:_after)?\(\);", body)
    assert at, name + " does not wait"
    before = body[:at.start()]
    assert MAY_STAND_BEFORE.fullmatch(before), (name, before)


@pytest.mark.parametrize("file,name,params,body", [k for k in KERNELS if k[0] in ("embed.cu", "balance.cu")],
                         ids=[k[1] for k in KERNELS if k[0] in ("embed.cu", "balance.cu")])
def test_inputs_are_not_promised_to_stand_still(file, name, params, body):
    """const __restrict__ says that nobody writes the data while the kernel runs, which lets the compiler read it through
    the incoherent cache and before the wait.  A kernel that starts while the one before it still writes its inputs
    cannot say so."""
    assert not re.findall(r"const\s+\w+\s*\*\s*__restrict__\s+(\w+)", params)
