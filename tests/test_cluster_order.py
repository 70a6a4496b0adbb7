"""Kernels whose CTAs read one another's shared memory: a CTA may leave once the others have read it. A relaxed arrival at the
cluster's barrier orders no earlier access, so that it must not be what says that the reads are done. Like the order of loads
behind a wait this is a property of the sources."""
import re

import pytest

from test_stream_order import SOURCES, code, kernels


def last_reads(body):
    """What follows the last load from another CTA's shared memory, up to the cluster's next wait."""
    at = body.rindex("ld.shared::cluster")
    return body[at:body.index("cluster_wait()", at)]


def reading():
    return [(f, n, b) for f in SOURCES for n, _, b in kernels(code(f)) if "ld.shared::cluster" in b]


def test_such_kernels_are_found():
    assert "paged_attn_kernel" in [n for _, n, _ in reading()]


@pytest.mark.parametrize("file,name,body", reading(), ids=[n for _, n, _ in reading()])
def test_the_arrival_behind_remote_reads_orders_them(file, name, body):
    arrivals = re.findall(r"\bcluster_arrive\w*\(\)", last_reads(body))
    assert arrivals == ["cluster_arrive()"], (file, name, arrivals)
