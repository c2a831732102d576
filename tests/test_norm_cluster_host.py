"""Layer norm's kernels and the shared memory of a cluster, by their source.

They reach other CTAs through RowSum, a device function.  Two things have to hold: a CTA is
known to have started before another sends to it; and a warp's reads of a stage are ordered before
the sends that let another thread fill the stage again, by all of its lanes and not the sending
ones alone (backward reads values of the residual that nothing it sends depends on)."""
import os
import re

import pytest

from test_cluster_start_host import CSRC, kernels, without_comments

# what touches another CTA's shared memory, and the row sums, which do so in a function of their own
REMOTE = re.compile(r"\b(map_rank|st_cluster\w*|ld_cluster|mbar_arrive_cluster)\s*\(|\bsum2?\s*\(\w+, warp, lane, a\.ctas\)")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return without_comments(f.read())


def sends_in_order(text):
    """Whether in RowSum a __syncwarp() stands between entering the cluster's branch and its sends."""
    branch = text.index("if constexpr (C::CLUSTER)", text.index("struct RowSum"))
    return 0 <= text.find("__syncwarp();", branch) < text.index("st_cluster_tx(", branch)


def starts_first(body):
    first = REMOTE.search(body)
    return first is not None and 0 <= body.find("cluster_arrive();") < body.find("cluster_wait();") < first.start()


def test_reads_of_a_stage_before_the_sends():
    assert sends_in_order(source("norm_rows.cuh"))


@pytest.mark.parametrize("name,kernel", [("norm_forward.cu", "k_norm_forward"), ("norm_backward.cu", "k_norm_backward"),
                                         ("ns_kernel.cuh", "k_ns")])
def test_every_cta_has_started(name, kernel):
    body = dict(kernels(source(name)))[kernel]
    assert starts_first(body)
    assert not starts_first(body.replace("cluster_wait();", "", 1).replace("cluster_arrive();", "", 1))


def test_no_kernel_is_missed():
    """Every kernel of the library that can run as a cluster is one of those that are looked at, here or in
    test_cluster_start_host."""
    found = set()
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh")):
            found |= {n for n, body in kernels(source(f)) if REMOTE.search(body) or "cluster_rank()" in body}
    assert found == {"k_linear", "k_skinny_dgrad", "k_ns", "k_norm_forward", "k_norm_backward"}
