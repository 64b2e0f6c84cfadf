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


def norm(lib, where, rows=T, ldx=K, ldr=K, ldh=K, ldy=K, xt=0, st=0):
    """Buffers by name at offsets in bytes, the others apart."""
    p = {n: at(FAR * (i + 1)) for i, n in enumerate(("X", "R", "w", "H", "Y", "Q", "SQ", "rstd"))}
    p.update({n: at(v) for n, v in where.items()})
    return lib.moe_norm(xt, p["X"], ldx, st, p["R"], ldr, 0, p["w"], 1e-6, rows, K, p["H"], ldh, p["Y"], ldy, p["Q"],
                        p["SQ"], 0, p["rstd"], None)


NORM = {
    "h_a_row_behind_r": dict(where=dict(R=0, H=2 * K)),
    "h_over_r_of_another_stride": dict(where=dict(R=0, H=0), ldr=WIDE),
    "h_over_x_of_another_type": dict(where=dict(X=0, H=0), st=1),
    "y_over_fp32_x": dict(where=dict(X=0, Y=0), xt=1),
    "y_into_x": dict(where=dict(X=0, Y=128), ldx=WIDE, ldy=WIDE),
    "codes_over_x": dict(where=dict(X=0, Q=0)),
    "y_over_w": dict(where=dict(w=0, Y=-(T - 1) * 2 * K)),
    "rstd_over_w": dict(where=dict(w=0, rstd=2 * K - 4)),
    "rstd_over_r": dict(where=dict(R=0, rstd=2 * T * K - 4)),
}


@pytest.mark.parametrize("name", sorted(NORM))
def test_norm_refuses_outputs_over_inputs(lib, name):
    assert norm(lib, **NORM[name]) == 1


def norm_backward(lib, where, rows=T, ldd=K, ldh=K, ldr=K, ldx=K, gt=0, st=0, wt=0):
    p = {n: at(FAR * (i + 1)) for i, n in enumerate(("dY", "H", "w", "rstd", "dR", "dX", "dw", "work"))}
    p.update({n: at(v) for n, v in where.items()})
    need = lib.moe_norm_work_bytes(rows, K)
    return lib.moe_norm_backward(gt, p["dY"], ldd, st, p["H"], ldh, wt, p["w"], p["rstd"], p["dR"], ldr, rows, K, p["dX"],
                                 ldx, p["dw"], p["work"], need, None)


NORM_BACKWARD = {
    "dx_a_row_behind_dr": dict(where=dict(dR=0, dX=2 * K)),
    "dx_over_h_of_another_stride": dict(where=dict(H=0, dX=0), ldh=WIDE),
    "dx_over_dy_of_another_type": dict(where=dict(dY=0, dX=0), gt=1),
    "dw_over_h": dict(where=dict(H=0, dw=2 * T * K - 16)),
    "dw_over_w": dict(where=dict(w=0, dw=0)),
    "dw_over_fp32_w": dict(where=dict(w=0, dw=0), wt=1),
    "work_over_rstd": dict(where=dict(work=0, rstd=T * K * 4 - 16)),
}


@pytest.mark.parametrize("name", sorted(NORM_BACKWARD))
def test_norm_backward_refuses_outputs_over_inputs(lib, name):
    assert norm_backward(lib, **NORM_BACKWARD[name]) == 1
