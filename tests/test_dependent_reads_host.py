"""How kernels that start before the kernel in front has ended read memory (CPU only).

The read-only load path (``ld.global.nc``: ``__ldg``, or a pointer that the compiler
may take for one) asks that nothing writes the memory during the kernel's whole
life.  A programmatic dependent may be resident while the kernel in front still
writes its inputs, so what it reads after its wait goes through ordinary loads or
loads past L1.  The fused GEMM and the NF4 GEMV use the read-only path for the frozen
weight alone: they start behind a rank-r kernel that has itself waited."""

import os
import re

import pytest

from quantized_rank_fine_b200 import build

READ_ONLY = re.compile(r"__ldg\s*\(|ld\.global\.nc|__restrict__")


def code(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", f.read()), flags=re.S)


@pytest.mark.parametrize("name", ["matvec.cu", "rmsnorm.cu", "skinny.cu", "xa_small.cu"])
def test_dependents_do_not_use_the_read_only_path(name):
    text = code(name)
    assert "grid_dependency_wait()" in text
    assert READ_ONLY.findall(text) == []


@pytest.mark.parametrize("name", ["gemm.cu", "gemv.cu"])
def test_only_the_frozen_weight_goes_through_it(name):
    reads = re.findall(r"__ldg\s*\(([^;]*);", code(name))
    assert reads and all(re.search(r"p\.dq_(?:codes|scales)", r) for r in reads)
