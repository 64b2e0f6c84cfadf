"""The slot map's buffers may not overlap: its blocks read the choices of others
while these write rows, so a map in place would race.  Refused before anything
is launched; runs on the CPU."""
import ctypes

import pytest

from moe_grouped_gemm_side_gb300 import binding as mb
from tests.test_binding_guards import i32

pytestmark = pytest.mark.cpu

BASE, STEP = 1 << 24, 1 << 20
T, k, E, CAP = 4096, 4, 8, 4096
N = T * k * 4                                       # bytes of the choices, and of the rows
WORK = 4 * E * 4                                    # four chunks of 4096 choices
BUFFERS = ["idx", "rows", "counts", "src", "work"]
SIZES = dict(idx=N, rows=N, counts=4 * E, src=4 * CAP, work=WORK)


def places(**moved):
    p = {b: BASE + i * STEP for i, b in enumerate(BUFFERS)}
    p.update(moved)
    return {b: ctypes.c_void_p(v) for b, v in p.items()}


def contiguous(lib, p):
    return lib.moe_slots_contiguous(p["idx"], T, k, E, 16, CAP, p["rows"], p["counts"], p["src"], p["work"], WORK, None,
                                    None)


def masked(lib, p):
    return lib.moe_slots_masked(p["idx"], T, k, E, CAP // E, p["rows"], p["counts"], p["src"], p["work"], WORK, None,
                                None)


PAIRS = [(a, b) for i, a in enumerate(BUFFERS) for b in BUFFERS[i + 1:]]


@pytest.mark.parametrize("call", [contiguous, masked])
@pytest.mark.parametrize("a,b", PAIRS)
def test_overlaps_are_refused(lib, call, a, b):
    at = BASE + 8 * STEP
    assert call(lib, places(**{a: at, b: at})) == 1
    # the last 16 bytes of one are the first of the other
    assert call(lib, places(**{a: at, b: at + SIZES[a] - 16})) == 1
    assert call(lib, places(**{b: at, a: at + SIZES[b] - 16})) == 1


def test_binding_refuses_a_map_in_place(monkeypatch, lib):
    monkeypatch.setattr(mb, "_on_device", lambda t: True)
    monkeypatch.setattr(mb, "_stream", lambda s: None)
    idx = i32(64, 2)
    with pytest.raises(mb.MoeGemmError) as err:
        mb.slots_contiguous(idx, idx, i32(8), 16, 256)
    assert err.value.code == 1
    with pytest.raises(mb.MoeGemmError) as err:
        mb.slots_masked(idx, i32(64, 2), i32(8), 16, src=idx.view(-1))
    assert err.value.code == 1
