"""Refusals of the operators around the grouped GEMMs: bad arguments come back
as error codes before anything is launched, and the binding refuses tensors
that the library would misread or overrun.  Runs on the CPU."""
import ctypes

import pytest
import torch

from moe_grouped_gemm_side_gb300 import binding as mb
from tests.test_abi import FAKE, MISALIGNED
from tests.test_binding_guards import StandIn, bf16, fake, i32, u8  # noqa: F401

pytestmark = pytest.mark.cpu

ODD = ctypes.c_void_p((1 << 20) + 1)


def caller(fn, args):
    def call(change):
        a = list(args)
        for i, v in change.items():
            a[i] = v
        return fn(*a)
    return call


def test_route_refusals(lib):
    # lt, logits, ld, bias, T, E, k, score, groups, top_groups, group_top, renorm, scale, idx, w, status, stream
    r = caller(lib.moe_route, [0, FAKE, 64, None, 4, 64, 8, 1, 1, 1, 1, 0, 1.0, FAKE, FAKE, None, None])
    assert r({0: 2}) == 1 and r({0: 7}) == 1           # logits as E4M3, unknown type
    assert r({1: None}) == 1
    assert r({2: 63}) == 1                              # rows overlap
    assert r({4: -1}) == 1 and r({5: 0}) == 1 and r({6: 0}) == 1
    assert r({6: 65}) == 2 and r({5: 16, 6: 17, 2: 16}) == 1     # k past 32, k past E
    assert r({5: 1025, 2: 1025}) == 2
    assert r({7: 0}) == 1 and r({7: 3}) == 1
    assert r({8: 0}) == 1 and r({8: 5}) == 1 and r({8: 64, 9: 1}) == 2
    assert r({8: 8, 9: 9}) == 1 and r({8: 8, 9: 0}) == 1
    assert r({10: 0}) == 1 and r({10: 3}) == 1
    assert r({12: float("nan")}) == 1 and r({12: float("inf")}) == 1
    assert r({13: None}) == 1 and r({14: None}) == 1
    assert r({13: ODD}) == 1 and r({14: ODD}) == 1 and r({1: ODD}) == 1 and r({3: ODD}) == 1
    assert r({4: 2 ** 30}) == 2                         # T * k past 2^31
    assert r({4: 0, 1: None, 13: None, 14: None}) == 0  # no tokens: nothing to do


def test_route_backward_refusals(lib):
    # lt, logits, ld, idx, dw, T, E, k, score, renorm, scale, dlogits, ldd, status, stream
    r = caller(lib.moe_route_backward, [1, FAKE, 64, FAKE, FAKE, 4, 64, 8, 2, 0, 1.0, FAKE, 64, None, None])
    assert r({0: 2}) == 1 and r({1: None}) == 1 and r({3: None}) == 1 and r({4: None}) == 1 and r({11: None}) == 1
    assert r({12: 63}) == 1 and r({8: 4}) == 1 and r({10: float("nan")}) == 1
    assert r({11: ctypes.c_void_p((1 << 20) + 2)}) == 1     # fp32 at a 2-byte address
    assert r({5: 0, 1: None, 3: None, 4: None, 11: None}) == 0


def test_slots_refusals(lib):
    # idx, T, k, E, align_q, rows_cap, rows, counts, src, work, work_bytes, status, stream
    r = caller(lib.moe_slots_contiguous, [FAKE, 64, 4, 8, 16, 512, FAKE, FAKE, None, None, 0, None, None])
    assert r({0: None}) == 1 and r({6: None}) == 1 and r({7: None}) == 1
    assert r({1: -1}) == 1 and r({2: 0}) == 1 and r({2: 33}) == 2 and r({3: 0}) == 1 and r({3: 1025}) == 2
    assert r({4: 0}) == 1 and r({5: 0}) == 1 and r({5: 2 ** 31}) == 1
    assert r({1: 2 ** 25}) == 2                         # 2^27 choices
    assert r({7: MISALIGNED}) == 1                      # the GEMMs want aligned counts
    need = lib.moe_slots_work_bytes(8192, 8)
    assert lib.moe_slots_work_bytes(4096, 8) == 0 and need == 2 * 8 * 4
    assert r({1: 2048}) == 1 and r({1: 2048, 9: FAKE, 10: need - 1}) == 1
    # idx, T, k, E, M_max, rows, counts, src, work, work_bytes, status, stream
    m = caller(lib.moe_slots_masked, [FAKE, 64, 4, 8, 64, FAKE, FAKE, None, None, 0, None, None])
    assert m({4: 0}) == 1 and m({4: 2 ** 29}) == 1 and m({0: None}) == 1 and m({3: 1025}) == 2


def test_dispatch_refusals(lib):
    # xt, X, ldx, SX, rows, T, k, K, at, A, SFA, rows_total, group_rows, CX, SCX, status, stream
    r = caller(lib.moe_dispatch, [0, FAKE, 256, None, FAKE, 4, 2, 256, 0, FAKE, None, 64, 64, None, None, None, None])
    assert r({0: 1}) == 1 and r({8: 1}) == 1            # fp32 is no row type
    assert r({1: None}) == 1 and r({4: None}) == 1 and r({9: None}) == 1
    assert r({2: 248}) == 1 and r({2: 260}) == 2        # rows overlap; stride not whole vectors
    assert r({7: 0}) == 1 and r({7: 252, 2: 256}) == 2
    assert r({0: 2, 3: None}) == 1                      # codes without scales
    assert r({8: 2}) == 1                               # E4M3 rows without scales
    assert r({8: 2, 10: FAKE, 7: 200, 2: 200}) == 2     # E4M3 wants whole blocks
    assert r({13: FAKE}) == 1 and r({14: FAKE}) == 1    # a checkpoint is codes and scales
    assert r({0: 2, 3: FAKE, 13: FAKE, 14: FAKE}) == 1  # of a bf16 source
    assert r({11: 0}) == 1 and r({11: 2 ** 31, 12: 2 ** 31}) == 1 and r({12: 48}) == 1 and r({12: 128}) == 1
    assert r({1: MISALIGNED}) == 1 and r({9: MISALIGNED}) == 1 and r({13: MISALIGNED, 14: FAKE}) == 1
    assert r({6: 33}) == 2 and r({7: 2 ** 25, 2: 2 ** 25}) == 2
    assert r({5: 0, 1: None, 4: None, 9: None}) == 0


def test_combine_refusals(lib):
    # D, rows, w, T, k, K, rows_total, ot, out, ldo, status, stream
    r = caller(lib.moe_combine, [FAKE, FAKE, None, 4, 2, 256, 64, 0, FAKE, 256, None, None])
    assert r({7: 2}) == 1 and r({0: None}) == 1 and r({1: None}) == 1 and r({8: None}) == 1
    assert r({5: 0}) == 1 and r({5: 252}) == 2 and r({9: 248}) == 1 and r({9: 260}) == 2 and r({6: 0}) == 1
    assert r({0: MISALIGNED}) == 1 and r({8: MISALIGNED}) == 1 and r({2: ODD}) == 1
    # gt, dout, ldd, D, rows, w, T, k, K, rows_total, dD, dw, status, stream
    b = caller(lib.moe_combine_backward, [0, FAKE, 256, FAKE, FAKE, None, 4, 2, 256, 64, FAKE, FAKE, None, None])
    assert b({0: 2}) == 1 and b({1: None}) == 1 and b({10: None}) == 1 and b({4: None}) == 1
    assert b({3: None}) == 1 and b({11: None}) == 1     # D and dw together or not at all
    assert b({2: 255}) == 1 and b({2: 260}) == 2 and b({8: 100, 2: 256}) == 2
    assert b({10: MISALIGNED}) == 1


def test_swiglu_refusals(lib):
    # H, rows_total, group_rows, N, src, out, Y, SFY, HC, SHC, stream
    r = caller(lib.moe_swiglu_save, [FAKE, 64, 64, 512, None, 1, FAKE, None, FAKE, FAKE, None])
    assert r({3: 384}) == 2 and r({3: 0}) == 1 and r({1: 0}) == 1 and r({2: 48}) == 1
    assert r({5: 0}) == 1 and r({5: 2}) == 1            # E4M3 output without scales
    for i in (0, 6, 8, 9):
        assert r({i: None}) == 1
    assert r({0: MISALIGNED}) == 1 and r({6: MISALIGNED}) == 1 and r({8: MISALIGNED}) == 1 and r({9: ODD}) == 1
    # dY, HC, SHC, rows_total, N, src, w, n, dH, Y, dw, status, stream
    b = caller(lib.moe_swiglu_backward, [FAKE, FAKE, FAKE, 64, 512, FAKE, FAKE, 8, FAKE, None, None, None, None])
    for i in (0, 1, 2, 8):
        assert b({i: None}) == 1
    assert b({4: 384}) == 2 and b({3: 0}) == 1 and b({7: -1}) == 1
    assert b({5: None}) == 1                            # weights without a map
    assert b({8: MISALIGNED}) == 1 and b({9: MISALIGNED}) == 1


def f32(*shape):
    return torch.zeros(shape, dtype=torch.float32)


def test_binding_accepts_exact_operands(fake):  # noqa: F811
    T, k, E, K, N = 6, 2, 4, 256, 512
    mb.route(f32(T, E), i32(T, k), f32(T, k), bias=f32(E))
    mb.route(bf16(T, 9)[:, 2:6], i32(T, k), f32(T, k), score="sigmoid")
    mb.route_backward(bf16(T, E), i32(T, k), f32(T, k), bf16(T, E))
    mb.slots_contiguous(i32(T, k), i32(T, k), i32(E), 16, 96, src=i32(96))
    mb.slots_masked(i32(T, k), i32(T, k), i32(E), 16, src=i32(64), work=u8(8))
    mb.dispatch(bf16(T, K), i32(T, k), bf16(96, K))
    mb.dispatch(bf16(T, K), i32(T, k), u8(E, 16, K), SFA=u8(E, K // 128, 16), CX=u8(T, K), SCX=u8(T, K // 128))
    mb.dispatch(u8(T, K), i32(T, k), bf16(96, K), SX=u8(T, K // 128))
    mb.combine(bf16(96, K), i32(T, k), f32(T, K), w=f32(T, k))
    mb.combine(bf16(E, 16, K), i32(T, k), bf16(T, K))
    mb.combine_backward(bf16(T, K), bf16(96, K), i32(T, k), f32(T, k), bf16(96, K), f32(T, k))
    mb.combine_backward(f32(T, K), None, i32(T, k), None, bf16(96, K), None)
    mb.swiglu_save(bf16(96, N), bf16(96, N // 2), u8(96, N), u8(96, N // 128), src=i32(96))
    mb.swiglu_save(bf16(E, 16, N), u8(E, 16, N // 2), u8(64, N), u8(64, N // 128), SFY=u8(E, N // 256, 16))
    mb.swiglu_backward(bf16(96, N // 2), u8(96, N), u8(96, N // 128), bf16(96, N))
    mb.swiglu_backward(bf16(96, N // 2), u8(96, N), u8(96, N // 128), bf16(96, N), w=f32(T, k), src=i32(96),
                       Y=bf16(96, N // 2), dw=f32(T, k))
    assert len(fake.calls) == 16


T, k, E, K, N = 6, 2, 4, 256, 512
REFUSED = {
    "logits_dtype": lambda: mb.route(u8(T, E), i32(T, k), f32(T, k)),
    "logits_strided": lambda: mb.route(f32(E, T).t(), i32(T, k), f32(T, k)),
    "logits_rows": lambda: mb.route(f32(T - 1, E), i32(T, k), f32(T, k)),
    "idx_dtype": lambda: mb.route(f32(T, E), i32(T, k).long(), f32(T, k)),
    "idx_strided": lambda: mb.route(f32(T, E), i32(T, 2 * k)[:, ::2], f32(T, k)),
    "w_short": lambda: mb.route(f32(T, E), i32(T, k), f32(T, k - 1)),
    "w_dtype": lambda: mb.route(f32(T, E), i32(T, k), bf16(T, 2 * k)),
    "bias_short": lambda: mb.route(f32(T, E), i32(T, k), f32(T, k), bias=f32(E - 1)),
    "score": lambda: mb.route(f32(T, E), i32(T, k), f32(T, k), score="tanh"),
    "dlogits_type": lambda: mb.route_backward(f32(T, E), i32(T, k), f32(T, k), bf16(T, 2 * E)),
    "dlogits_shape": lambda: mb.route_backward(f32(T, E), i32(T, k), f32(T, k), f32(T, E + 1)),
    "dw_short": lambda: mb.route_backward(f32(T, E), i32(T, k), f32(T - 1, k), f32(T, E)),
    "rows_short": lambda: mb.slots_contiguous(i32(T, k), i32(T - 1, k), i32(E), 16, 96),
    "src_short": lambda: mb.slots_contiguous(i32(T, k), i32(T, k), i32(E), 16, 96, src=i32(95)),
    "src_masked_short": lambda: mb.slots_masked(i32(T, k), i32(T, k), i32(E), 16, src=i32(63)),
    "counts_dtype": lambda: mb.slots_masked(i32(T, k), i32(T, k), i32(E).long(), 16),
    "x_shape": lambda: mb.dispatch(bf16(T, K - 128), i32(T, k), bf16(96, K)),
    "x_dtype": lambda: mb.dispatch(f32(T, K), i32(T, k), bf16(96, K)),
    "no_sx": lambda: mb.dispatch(u8(T, K), i32(T, k), bf16(96, K)),
    "no_sfa": lambda: mb.dispatch(bf16(T, K), i32(T, k), u8(96, K)),
    "sfa_short": lambda: mb.dispatch(bf16(T, K), i32(T, k), u8(96, K), SFA=u8(K // 128, 80)),
    "half_a_checkpoint": lambda: mb.dispatch(bf16(T, K), i32(T, k), bf16(96, K), CX=u8(T, K)),
    "short_checkpoint": lambda: mb.dispatch(bf16(T, K), i32(T, k), bf16(96, K), CX=u8(T, K), SCX=u8(T, 1)),
    "a_strided": lambda: mb.dispatch(bf16(T, K), i32(T, k), bf16(96, 2 * K)[:, :K]),
    "out_shape": lambda: mb.combine(bf16(96, K), i32(T, k), bf16(T, K + 8)),
    "out_dtype": lambda: mb.combine(bf16(96, K), i32(T, k), u8(T, K)),
    "d_dtype": lambda: mb.combine(f32(96, K), i32(T, k), bf16(T, K)),
    "combine_w_short": lambda: mb.combine(bf16(96, K), i32(T, k), bf16(T, K), w=f32(T, 1)),
    "d_short": lambda: mb.combine_backward(bf16(T, K), bf16(95, K), i32(T, k), None, bf16(96, K), f32(T, k)),
    "dout_shape": lambda: mb.combine_backward(bf16(T + 1, K), None, i32(T, k), None, bf16(96, K), None),
    "y_short": lambda: mb.swiglu_save(bf16(96, N), bf16(95, N // 2), u8(96, N), u8(96, N // 128)),
    "hc_short": lambda: mb.swiglu_save(bf16(96, N), bf16(96, N // 2), u8(96, N - 1), u8(96, N // 128)),
    "shc_short": lambda: mb.swiglu_save(bf16(96, N), bf16(96, N // 2), u8(96, N), u8(95, N // 128)),
    "no_sfy": lambda: mb.swiglu_save(bf16(96, N), u8(96, N // 2), u8(96, N), u8(96, N // 128)),
    "map_short": lambda: mb.swiglu_save(bf16(96, N), bf16(96, N // 2), u8(96, N), u8(96, N // 128), src=i32(95)),
    "dy_short": lambda: mb.swiglu_backward(bf16(95, N // 2), u8(96, N), u8(96, N // 128), bf16(96, N)),
    "dh_dtype": lambda: mb.swiglu_backward(bf16(96, N // 2), u8(96, N), u8(96, N // 128), f32(96, N)),
    "w_and_dw_differ": lambda: mb.swiglu_backward(bf16(96, N // 2), u8(96, N), u8(96, N // 128), bf16(96, N),
                                                  w=f32(T, k), src=i32(96), dw=f32(T - 1, k)),
}


@pytest.mark.parametrize("case", sorted(REFUSED))
def test_binding_refusals(fake, case):  # noqa: F811
    with pytest.raises((ValueError, TypeError)):
        REFUSED[case]()
    assert fake.calls == []
