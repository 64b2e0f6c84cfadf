"""Rows that a call writes may not share bytes with rows that it reads, but for the
calls in place that the interface names: blocks read what others write.  Refused
before anything is launched; runs on the CPU."""
import ctypes

import pytest

pytestmark = pytest.mark.cpu

AT, FAR = 1 << 30, 1 << 24
T, K, N, WIDE = 40, 256, 128, 640


def at(offset):
    return ctypes.c_void_p(AT + offset)


def adapters(lib, x, base, y, ldx=K, ldb=N, ldy=N, rows=T):
    """Offsets in bytes of X, base (None: Y) and Y; the others lie apart."""
    other = [at(FAR * i) for i in range(1, 7)]
    return lib.moe_adapters(at(x), ldx, other[0], other[1], None, other[2], other[3], other[4], rows, 3, 16, K, N, 64, 16,
                            None if base is None else at(base), ldb, at(y), ldy, None, None)


# X, base, Y, their strides
SHARED = {
    "y_behind_base": (8 * FAR, 0, (T - 1) * N * 2, K, N, N),          # the last row is the first
    "y_before_base": (8 * FAR, (T * N - 8) * 2, 0, K, N, N),          # eight columns
    "columns": (8 * FAR, 0, 64 * 2, K, WIDE, WIDE),                   # half of every row
    "columns_before": (8 * FAR, 64 * 2, 0, K, WIDE, WIDE),
    "columns_rows_on": (8 * FAR, 0, (5 * WIDE + 120) * 2, K, WIDE, WIDE),
    "around_the_stride": (8 * FAR, 0, (WIDE - 120) * 2, K, WIDE, WIDE),       # a row of Y reaches the next of base
    "other_stride": (8 * FAR, 0, 5 * WIDE * 2, K, N, WIDE),
    "other_stride_far": (8 * FAR, 200 * 2, 0, K, WIDE, 2 * WIDE + 8),
    "y_over_x": (0, 8 * FAR, 0, K, N, K),
    "y_in_x": (0, 8 * FAR, 128 * 2, WIDE, N, WIDE),
    "y_in_x_in_place": (0, None, (T - 1) * K * 2, K, 0, N),
}


@pytest.mark.parametrize("name", sorted(SHARED))
def test_adapters_refuse_rows_that_share_bytes(lib, name):
    x, base, y, ldx, ldb, ldy = SHARED[name]
    assert adapters(lib, x, base, y, ldx, ldb, ldy) == 1
