"""Copies and products in flight when a block gives up its waits land before its
memory goes, whatever limit a program has set for the waits: drains have a time of
their own.  Reads the sources; runs on the CPU."""
import re

import pytest

from tests.test_ops_sources import source, sources

pytestmark = pytest.mark.cpu


def test_drains_do_not_hang_on_the_wait_limit():
    seen = 0
    for name in sources():
        text = source(name)
        for m in re.finditer(r"(?<!bool )\bwait_drain\(([^;]*)\);", text):
            seen += 1
            until = m.group(1).rsplit(",", 1)[1].strip()
            if re.fullmatch(r"\w+\)?", until):
                until = re.findall(r"\b%s = ([^;]*);" % until.rstrip(")"), text[:m.start()])[-1]
            assert "kDrainNs" in until and "wait_ns" not in until, (name, until)
    assert seen >= 8
