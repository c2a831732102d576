"""Shared memory of another CTA of a cluster may be touched only once that CTA is known to have
started: in every kernel a completed cluster barrier stands before the first such access."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fsdp_sharded_state_gb300", "csrc")
REMOTE = re.compile(r"\b(map_rank|st_cluster4?|ld_cluster|mbar_arrive_cluster)\s*\(")


def without_comments(text):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def kernels(text):
    """(name, body) of the __global__ functions."""
    for m in re.finditer(r"__global__", text):
        name = re.search(r"\b(k_\w+)\s*\(", text[m.end():])
        at = start = text.index("{", text.index(")", m.end() + name.end()))
        depth = 0
        while True:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
            if depth == 0:
                break
        yield name.group(1), text[start:at]


def remote_kernels():
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            for name, body in kernels(without_comments(f.read())):
                if REMOTE.search(body):
                    found.append(pytest.param(body, id=f"{os.path.basename(path)}:{name}"))
    return found


@pytest.mark.parametrize("body", remote_kernels())
def test_barrier_before_remote_shared_memory(body):
    arrive, wait = body.find("cluster_arrive();"), body.find("cluster_wait();")
    assert 0 <= arrive < wait < REMOTE.search(body).start()


def test_kernels_are_found():
    assert {p.id.split(":")[1] for p in remote_kernels()} >= {"k_linear", "k_skinny_dgrad"}
