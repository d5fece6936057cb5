"""A CTA may touch the shared memory of another of its cluster only once that one is known to run: a
kernel that does so has waited at the cluster's barrier before. (An access that comes too early cannot be
made to happen on demand, so the order is looked for in the source.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gated_deltanet_linear_scan_gb300", "csrc")
REMOTE = re.compile(r"\b(in_cta|ld_shared_cluster)\(")
WAIT = re.compile(r"\b(cluster_wait_acquire|cluster_sync)\(\)")


def kernels(text):
    """(name, body) of every kernel: from its name to the closing brace at the line's start."""
    for m in re.finditer(r"__global__.*?\b(\w+)\(const ", text, re.S):
        yield m.group(1), text[m.end():text.index("\n}\n", m.end())]


def without_lambdas(body):
    """The body less its lambdas that are only defined here: they run where they are called."""
    return re.sub(r"\n    auto \w+ = \[[^\n]*\{\n.*?\n    };", "", body, flags=re.S)


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith(".cu")))
def test_clusters_wait_before_remote_accesses(name):
    text = open(os.path.join(CSRC, name)).read()
    if not REMOTE.search(text):
        return
    seen = 0
    for kernel, body in kernels(text):
        body = without_lambdas(body)
        first = REMOTE.search(body)
        if first is None:
            continue
        seen += 1
        wait = WAIT.search(body)
        assert wait and wait.start() < first.start(), f"{kernel} of {name} reaches another CTA before it waits"
    assert seen > 0, f"no kernel of {name} was looked at"
