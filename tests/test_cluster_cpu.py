"""Thread-block clusters, checked in the kernels' source (no GPU): what goes wrong
here is a matter of order that a run seldom shows."""
import os
import re

import pytest

from depth_wise_attention_gb300.build import CSRC

# a write into another CTA's shared memory, and a wait for every CTA of the cluster
REMOTE = r"st\.shared::cluster|st_async|map_shared_rank|mapa_u32|cm_send_sum\("
WAIT = r"barrier\.cluster\.wait|cluster\.sync\(\)|cm_cluster_sync\(\)|cluster_wait_started\(\)"


def kernels(name):
    """(kernel, body) of a source file, comments taken out."""
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"/\*.*?\*/|//[^\n]*", "", text, flags=re.S)
    for m in re.finditer(r"__global__([^;{]*)\{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield re.findall(r"(\w+)\s*\(", m.group(1))[-1], text[m.end():at]


@pytest.mark.parametrize("name", ["cache_read_few.cu", "cache_read_mma.cuh", "depth_read_decode.cuh", "msar.cu",
                                  "msar_phase1.cu", "msar_tile.cu"])
def test_no_write_into_a_cta_that_may_not_run_yet(name):
    """A CTA's shared memory may be written by others of its cluster only once it runs, and being
    scheduled with them does not say so: a cluster wait comes before the first such write."""
    found = 0
    for kernel, body in kernels(name):
        first = re.search(REMOTE, body)
        if first is None:
            continue
        found += 1
        wait = re.search(WAIT, body)
        assert wait is not None and wait.start() < first.start(), kernel
    assert found


def test_sums_are_sent_by_a_cta_that_has_not_given_up():
    """A CTA of the tensor-core read of quantised rows that gave up runs on without waiting; what it would send the
    others then belongs to no item that they wait for.  And the last cluster barrier alone does not say that
    what was sent has landed."""
    for kernel, body in kernels("cache_read_mma.cuh"):
        for m in re.finditer(r"cm_send_sum\(", body):
            assert body[:m.start()].rstrip().endswith("if (send)"), kernel
        send = re.search(r"const bool send = ([^;]*);", body)
        assert send is not None and "cm_aborted(flag)" in send.group(1), kernel
    text = open(os.path.join(CSRC, "cache_read_mma.cuh")).read()
    leave = text[text.index("void cm_leave_cluster("):]
    leave = leave[:leave.index("\n}\n")]
    assert leave.count("cm_cluster_sync();") == 2 and "globaltimer" not in leave
