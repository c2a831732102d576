"""Programmatic dependent launches, by the kernels' source: every kernel waits for the grid before it,
and one that lets the next start early does so only after its own wait."""
import os

import pytest

from test_cluster_start_host import CSRC, kernels, without_comments


PLAIN = {"k_clip_coop", "k_wait_selftest"}       # launched without the attribute: the stream's order holds for them


def all_kernels():
    found = []
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh")):
            with open(os.path.join(CSRC, f)) as h:
                for name, body in kernels(without_comments(h.read())):
                    if name not in PLAIN:
                        found.append(pytest.param(body, id=f"{f}:{name}"))
    return found


@pytest.mark.parametrize("body", all_kernels())
def test_waits_before_it_triggers(body):
    # the staged kernels are a call of run_pipeline, which waits
    wait, trigger = max(body.find("pdl_wait();"), body.find("run_pipeline(")), body.find("pdl_trigger();")
    assert wait >= 0 and (trigger < 0 or trigger > wait)
    assert "launch_dependents" not in body       # by pdl_trigger() alone


def test_the_pipeline_waits():
    with open(os.path.join(CSRC, "pipeline.cuh")) as f:
        text = without_comments(f.read())
    assert "pdl_wait();" in text[text.index("run_pipeline("):]


def test_kernels_that_trigger():
    assert {p.id.split(":")[1] for p in all_kernels() if "pdl_trigger" in p.values[0]} == {"k_ns", "k_ns_squares", "k_ns_pack", "k_muon_momentum"}
