"""A block's shared memory may be reached by the other blocks of its cluster only
once it is known to run: every kernel that reads or writes there has a cluster
barrier before its first access.  No run shows the lack of one, so this reads the
sources; runs on the CPU.  The barriers' aligned form also wants a warp's lanes
together, which they may not be behind a loop or a branch of their own."""
import re

import pytest

from tests.test_ops_sources import bodies, source, sources

pytestmark = pytest.mark.cpu

BARRIER = re.compile(r"\bcluster_(?:sync|wait)\(\)|barrier\.cluster\.wait")
REMOTE = re.compile(r"\bmapa_shared\(|\bmapa\.shared::cluster")


def test_no_remote_access_before_a_cluster_barrier():
    seen = 0
    for name in sources():
        for fn, body in bodies(source(name)):
            at = REMOTE.search(body)
            if at is None or fn == "mapa_shared":
                continue
            seen += 1
            barrier = BARRIER.search(body)
            assert barrier is not None and barrier.start() < at.start(), (name, fn)
    assert seen >= 4


@pytest.mark.parametrize("name", ["adapters.cu", "balance.cu"])
def test_lanes_meet_before_a_cluster_barrier(name):
    """Behind the last closing brace (or a statement under an if) before an aligned
    cluster barrier, the warp or the block meets."""
    seen = 0
    for fn, body in bodies(source(name)):
        for m in re.finditer(r"\bcluster_(?:sync|wait|arrive)\(\);", body):
            before = body[:m.start()]
            since = before[before.rfind("}") + 1:]
            if "}" not in before and not re.search(r"\b(?:if|for|while)\b", before):
                continue                                  # the kernel's start
            seen += 1
            assert re.search(r"__sync(?:warp|threads)\(\);|\bcluster_arrive\(\);", since), (name, fn, since)
    assert seen >= 2
