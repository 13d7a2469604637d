"""Stores into another CTA's shared memory, read from the kernels' sources (CPU only).

A CTA of a thread-block cluster may be written to by its peers only once it has
started.  A barrier of the whole cluster before the first such store says so; one
after the stores only says that they have landed.  Whether a peer starts late is not
in a test's hands, so the order of the two is checked where it is written."""

import os
import re

import pytest

from quantized_rank_fine_b200 import build

REMOTE = re.compile(r"\b(?:st_shared_cluster\w*|mbar_arrive_cluster|mbar_arrive_remote)\s*\(")
BARRIER = re.compile(r"\b(?:cluster_started_wait|cluster_sync)\s*\(\s*\)")


def remote_writes(source):
    """(kernel, whether the cluster has met before) for every write to a peer in the kernels of a source text."""
    text = re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", source), flags=re.S)
    for m in REMOTE.finditer(text):
        at = text.rfind("__global__", 0, m.start())
        name = re.search(r"\b(\w+_kernel)\s*\(", text[at:])
        before = text[at:m.start()]
        waits = [b.group(0) for b in BARRIER.finditer(before)]
        met = bool(waits) and ("cluster_sync" in waits[0] or "cluster_started_arrive()" in before)
        yield (name.group(1) if name else "?"), met


def kernels_with_remote_writes():
    found = {}
    for src in build.SOURCES:
        with open(os.path.join(build.CSRC, src)) as f:
            for name, met in remote_writes(f.read()):
                found[src, name] = found.get((src, name), True) and met
    return found


FOUND = kernels_with_remote_writes()


def test_the_kernels_that_write_to_peers_are_found():
    assert {k for _, k in FOUND} >= {"skinny_tc_kernel", "xa_small_kernel", "nf4_gemv_kernel", "matvec_kernel",
                                     "rmsnorm_bwd_kernel"}


@pytest.mark.parametrize("src,kernel", sorted(FOUND))
def test_cluster_has_started_before_the_first_write(src, kernel):
    assert FOUND[src, kernel], f"{src}: {kernel} writes to a peer before a barrier has shown that it has started"


def test_the_check_sees_a_missing_barrier():
    body = "__global__ void a_kernel(int p) {{ {} st_shared_cluster_f32(x, v); cluster_sync(); }}"
    assert dict(remote_writes(body.format(""))) == {"a_kernel": False}
    assert dict(remote_writes(body.format("// cluster_sync();\n"))) == {"a_kernel": False}
    assert dict(remote_writes(body.format("cluster_started_wait();"))) == {"a_kernel": False}
    assert dict(remote_writes(body.format("cluster_started_arrive(); cluster_started_wait();"))) == {"a_kernel": True}
