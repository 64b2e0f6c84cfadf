"""What the binding hands the library for the operators' row buffers: the groups
of E4M3 scales come from shapes that agree with each other, and anything else
is refused.  Runs on the CPU against a stand-in that records arguments."""
import pytest
import torch

from moe_grouped_gemm_side_gb300 import binding as mb
from tests.test_binding_guards import bf16, i32, u8

pytestmark = pytest.mark.cpu


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def f(*args):
            self.calls.append((name, args))
            return 0
        return f


@pytest.fixture
def lib_calls(monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(mb, "load", lambda path=None: lib)
    monkeypatch.setattr(mb, "_on_device", lambda t: True)
    monkeypatch.setattr(mb, "_stream", lambda s: None)
    return lib.calls


T, k, E, M, K, N = 6, 2, 4, 16, 256, 768
R = E * M


def dispatch(A, SFA):
    mb.dispatch(bf16(T, K), i32(T, k), A, SFA=SFA)


def save(H, SFY):
    R = H.numel() // N
    mb.swiglu_save(H, u8(*H.shape[:-1], N // 2), u8(R, N), u8(R, N // 128), SFY=SFY)


# rows, scales, and the (rows_total, group_rows) that they mean
LAYOUTS = [((R,), (1, R), (R, R)), ((R,), (R,), (R, R)), ((E, M), (E, M), (R, M)), ((1, R), (R,), (R, R)),
           ((R,), (E, M), (R, M)), ((R,), (2, R // 2), (R, R // 2))]


def scale_shape(groups, blocks):
    return groups[:-1] + (blocks, groups[-1])


@pytest.mark.parametrize("rows,groups,want", LAYOUTS)
def test_groups_of_scales(lib_calls, rows, groups, want):
    dispatch(u8(*rows, K), u8(*scale_shape(groups, K // 128)))
    save(bf16(*rows, N), u8(*scale_shape(groups, N // 256)))
    (n0, a0), (n1, a1) = lib_calls
    assert n0 == "moe_dispatch" and a0[11:13] == want
    assert n1 == "moe_swiglu_save" and a1[1:3] == want


# scales of enough bytes in a shape that contradicts the rows' layout
WRONG = [((E, M), (1, R)), ((E, M), (R,)), ((E, M), (M, E)), ((E, M), (E, 2 * M)), ((R,), (E, 2 * M)), ((R,), (2 * R,)),
         ((E, M), (2 * E, M))]


@pytest.mark.parametrize("rows,groups", WRONG)
def test_scales_that_contradict_the_rows(lib_calls, rows, groups):
    with pytest.raises(ValueError):
        dispatch(u8(*rows, K), u8(*scale_shape(groups, K // 128)))
    with pytest.raises(ValueError):
        save(bf16(*rows, N), u8(*scale_shape(groups, N // 256)))
    assert lib_calls == []


@pytest.mark.parametrize("shape", [(R * (K // 128),), (E, M, K // 128), (E, K // 128, M, 1), (R, K // 128)])
def test_scales_of_another_form(lib_calls, shape):
    with pytest.raises(ValueError):
        dispatch(u8(E, M, K), u8(*shape))
    with pytest.raises(ValueError):
        dispatch(u8(R, K), u8(*shape))
    assert lib_calls == []


# the rows are counted from the first dimensions, so [C] would be C rows of C
# columns and [a, b, c, C] a * b rows of C: the calls would run past the first
# buffer, or leave rows of the second out
NOT_ROWS = {
    "dispatch": lambda s: mb.dispatch(bf16(T, K), i32(T, k), bf16(*s, K)),
    "dispatch_e4m3": lambda s: mb.dispatch(bf16(T, K), i32(T, k), u8(*s, K), SFA=u8(K // 128, 256)),
    "combine": lambda s: mb.combine(bf16(*s, K), i32(T, k), bf16(T, K)),
    "combine_backward": lambda s: mb.combine_backward(bf16(T, K), None, i32(T, k), None, bf16(*s, K), None),
    "swiglu_save": lambda s: mb.swiglu_save(bf16(*s, K), bf16(256, K // 2), u8(256, K), u8(256, K // 128)),
    "swiglu_backward": lambda s: mb.swiglu_backward(bf16(256, K // 2), u8(256, K), u8(256, K // 128), bf16(*s, K)),
}


@pytest.mark.parametrize("shape", [(), (2, 2, 4)], ids=["1d", "4d"])
@pytest.mark.parametrize("call", sorted(NOT_ROWS))
def test_row_buffers_of_another_form(lib_calls, call, shape):
    with pytest.raises(ValueError):
        NOT_ROWS[call](shape)
    assert lib_calls == []


F16, I16, I8 = torch.float16, torch.int16, torch.int8
BYTES = [torch.float32, F16, torch.bfloat16, I16, I8, torch.bool]


def like(dtype, *shape):
    return torch.zeros(shape, dtype=dtype)


# an operand of 8-bit codes or scales in turn, of more than enough bytes in another type
TYPED = {
    "SX": lambda d: mb.dispatch(u8(T, K), i32(T, k), bf16(R, K), SX=like(d, T, K // 128)),
    "SFA": lambda d: mb.dispatch(bf16(T, K), i32(T, k), u8(R, K), SFA=like(d, K // 128, R)),
    "CX": lambda d: mb.dispatch(bf16(T, K), i32(T, k), bf16(R, K), CX=like(d, T, K), SCX=u8(T, K // 128)),
    "SCX": lambda d: mb.dispatch(bf16(T, K), i32(T, k), bf16(R, K), CX=u8(T, K), SCX=like(d, T, K // 128)),
    "HC": lambda d: mb.swiglu_save(bf16(R, N), bf16(R, N // 2), like(d, R, N), u8(R, N // 128)),
    "SHC": lambda d: mb.swiglu_save(bf16(R, N), bf16(R, N // 2), u8(R, N), like(d, R, N // 128)),
    "SFY": lambda d: mb.swiglu_save(bf16(R, N), u8(R, N // 2), u8(R, N), u8(R, N // 128), SFY=like(d, N // 256, R)),
    "backward HC": lambda d: mb.swiglu_backward(bf16(R, N // 2), like(d, R, N), u8(R, N // 128), bf16(R, N)),
    "backward SHC": lambda d: mb.swiglu_backward(bf16(R, N // 2), u8(R, N), like(d, R, N // 128), bf16(R, N)),
}


@pytest.mark.parametrize("operand", sorted(TYPED))
def test_types_of_codes_and_scales(lib_calls, operand):
    own = torch.float8_e4m3fn if operand.split()[-1] in ("CX", "HC") else torch.float8_e8m0fnu
    other = torch.float8_e8m0fnu if own is torch.float8_e4m3fn else torch.float8_e4m3fn
    for dtype in BYTES + [other]:
        with pytest.raises(TypeError):
            TYPED[operand](dtype)
    assert lib_calls == []
    TYPED[operand](torch.uint8)
    TYPED[operand](own)
    assert len(lib_calls) == 2
