"""What the vocabulary operators' kernels have to keep to and no result shows, read from their text."""
import os
import re

import pytest

import lm_head_vocab_gb300._lib as L

CSRC = os.path.join(os.path.dirname(L.__file__), "csrc")


def kernels(name):
    """Name and body of each __global__ function of a source file, without comments."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    text = re.sub(r"__launch_bounds__\((?:[^()]|\([^()]*\))*\)", "", text)
    for m in re.finditer(r"__global__\s+void\s+(\w+)\s*\([^{;]*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[m.end():i]


def test_kernels_are_found():
    assert {"cluster_sort_kernel", "token_sum_kernel"} <= {n for n, _ in kernels("embedding.cu")}


@pytest.mark.parametrize("source", ["embedding.cu", "beam_step.cu", "beam_reorder.cu"])
def test_a_cluster_has_started_before_its_shared_memories_are_written(source):
    # a store to a block of the cluster that has not begun to run is lost or worse: a cluster
    # barrier is passed before the first one
    for name, body in kernels(source):
        if "dsmem_map" not in body:
            continue
        first = body.index("dsmem_map")
        barriers = [body.find(b) for b in ("cluster_sync_all()", "cluster_wait()") if b in body]
        assert barriers and min(barriers) < first, name
        if "cluster_wait()" in body:
            assert 0 <= body.find("cluster_arrive_relaxed()") < body.index("cluster_wait()"), name
