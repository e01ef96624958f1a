"""Rules of the memory model that the recurrence's kernels keep and that no run shows reliably when
they are broken (the hardware mostly forgives it), checked in the source."""

import os
import re

from top_routing_grouped_gemm_gb300 import build as B


def source(name):
    """The code of a file, without its comments."""
    with open(os.path.join(B.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(code, head):
    """The text from `head` to the end of the block of braces that follows it."""
    at = code.index(head)
    start = end = code.index("{", code.index(")", at))
    depth = 0
    while True:
        depth += {"{": 1, "}": -1}.get(code[end], 0)
        end += 1
        if depth == 0:
            return code[start:end]


def test_barriers_that_other_blocks_complete_are_waited_for_at_cluster_scope():
    """The pairs' bytes and the barrier's completion come from other blocks of the cluster, so the
    wait has to acquire at the cluster's scope, which the plain form does not."""
    code = source("linear_recurrence.cu")
    waits = re.findall(r"(\w+)(?:<[^>]*>)?\(&\w+\.received\[", code)
    waits = [w for w in waits if "wait" in w]
    assert waits == ["wait_for_cluster"]
    assert "mbar_wait_cluster(" in body(code, "wait_for_cluster(uint64_t*")


def test_warps_converge_before_the_clusters_barriers():
    """barrier.cluster in its .aligned form is for warps whose threads run it together; before the
    first wait one thread of a warp has copied tiles on its own."""
    code = source("linear_recurrence.cu")
    for name in ("cluster_arrive", "cluster_wait"):
        text = body(code, f"void {name}(")
        assert text.index("__syncwarp();") < text.index("barrier.cluster.")
    # and nothing goes around the two
    assert len(re.findall(r"barrier\.cluster\.(?:arrive|wait)", code)) == 2


def test_kernels_set_up_early_read_through_the_coherent_path():
    """A kernel that is set up while the one before it ends is alive while its inputs may still be
    written, which loads of data that is read-only for a kernel's life (ld.global.nc) rule out."""
    early = [f for f in sorted(os.listdir(B.CSRC)) if '#include "overlap.cuh"' in source(f)]
    assert {"gdr_step.cu", "linear_recurrence.cu", "qk_norm_rope.cu"} <= set(early)
    for name in early:
        code = source(name)
        assert not re.search(r"__ldg\b|\.nc\b|__restrict__", code), name
