"""A CTA's shared memory may be touched by others of its cluster only once all
of them have started.  No run shows a missing wait reliably, so this reads the
sources: a kernel's first remote access comes after its cluster wait, whose
arrival is the kernel's start."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lfsr_seeded_moe_b200", "csrc")


def _body(source, kernel):
    """The text between a kernel's braces, without comments."""
    with open(os.path.join(CSRC, source)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index("{", re.search(r"\bvoid\b[^;{}]*\b%s\(" % kernel, text).end())
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i]
    raise AssertionError(f"{kernel} has no end")


@pytest.mark.parametrize("source,kernel,remote", [
    ("sample.cu", "sample_kernel", "map_shared_rank"),
    ("balance.cu", "balance_finish_kernel", "finish("),
])
def test_the_cluster_runs_before_the_first_remote_access(source, kernel, remote):
    body = _body(source, kernel)
    order = [body.find(s) for s in ("cluster_arrive()", "griddepcontrol.wait", "cluster_wait()", remote)]
    assert -1 not in order and order == sorted(order), order
