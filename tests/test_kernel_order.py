"""What the sources say of the order in which a kernel takes what other kernels wait for. (A kernel that took it too
early could wait for ever, so no test runs one that does.)"""

import glob
import os
import re

import pytest

from conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "descriptor_build_gb300", "csrc", "*.cu*")))


def kernels(text):
    """The text of each kernel, up to the next one's beginning."""
    begins = [m.start() for m in re.finditer(r"__global__", text)]
    return [text[a:b] for a, b in zip(begins, begins[1:] + [len(text)])]


def test_tensor_memory_is_taken_after_the_kernels_before():
    """A CTA that has columns of tensor memory and waits for the kernels before it keeps the columns from their CTAs that
    have not begun: neither goes on. So the wait comes first."""
    found = 0
    for path in SOURCES:
        with open(path) as f:
            for kernel in kernels(f.read()):
                if "tcgen05.alloc" in kernel:
                    found += 1
                    assert "wait_for_prerequisites();" in kernel[:kernel.index("tcgen05.alloc")], path
    assert found


@pytest.mark.parametrize("call", ["dependents_may_launch();", "tcgen05.dealloc"])
def test_what_is_taken_is_given_back(call):
    for path in SOURCES:
        with open(path) as f:
            for kernel in kernels(f.read()):
                if "tcgen05.alloc" in kernel:
                    assert kernel.count(call) == 1, path


def test_a_wait_that_runs_out_is_told_in_the_status_too():
    """A kernel of attention that gives up waiting says so in the counters, and that no request is a valid one."""
    told = 0
    for path in SOURCES:
        with open(path) as f:
            for kernel in kernels(f.read()):
                if "DB_ERR_TIMEOUT" in kernel and "attention_" in kernel:
                    told += 1
                    assert "status[i] = DB_PAGE_INVALID" in kernel[kernel.index("DB_ERR_TIMEOUT"):], path
    assert told
