"""Layer norm's kernels and the shared memory of a cluster, by their source.

A warp's reads of a stage are ordered before the sends that let another thread fill the stage
again, by all of its lanes and not the sending ones alone: backward reads values of the
residual that nothing it sends depends on."""
import os

from test_cluster_start_host import CSRC, without_comments


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return without_comments(f.read())


def sends_in_order(text):
    """Whether in RowSum a __syncwarp() stands between entering the cluster's branch and its sends."""
    branch = text.index("if constexpr (C::CLUSTER)", text.index("struct RowSum"))
    return 0 <= text.find("__syncwarp();", branch) < text.index("st_cluster_tx(", branch)


def test_reads_of_a_stage_before_the_sends():
    assert sends_in_order(source("norm_rows.cuh"))
