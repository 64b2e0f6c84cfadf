"""A block's shared memory may be reached by the other blocks of its cluster only
once it is known to run: every kernel that reads or writes there has a cluster
barrier before its first access.  No run shows the lack of one, so this reads the
sources; runs on the CPU."""
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
