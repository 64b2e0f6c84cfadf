"""Adapters at the edges of what their interface allows, on the GPU.  Tolerances as
in the operator's own tests."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_side_gb300 import binding as mb
from tests import ops_util as ou
from tests.test_gpu_u_adapters import BF16, bf16, check, slot_map, want64

pytestmark = pytest.mark.gpu


def test_adapters_of_prompts_give_up_their_waits(cuda):
    """With a limit of a nanosecond the waits for a contraction of 786 MB, 100 us at
    least, end at their first look: the call reports it, the context stays usable and
    the next call has its results."""
    T, E, r, K, N = 3000, 1, 8, 131072, 256
    rng = np.random.default_rng(21)
    X = torch.randn(T, K, device=cuda, generator=torch.Generator(cuda).manual_seed(1)).to(BF16)
    base = bf16(rng, (T, N), 1.0, cuda)
    A, B = bf16(rng, (E, r, K), K ** -0.5, cuda), bf16(rng, (E, N, r), r ** -0.5, cuda)
    idx, rows, src = slot_map(np.zeros(T, dtype=np.int64), E, 128, cuda)
    st = ou.status_word(cuda)
    want, Y = torch.empty_like(base), torch.empty_like(base)
    mb.adapters(X, A, B, want, idx, rows, src, 128, base=base, status=st)
    assert st.item() == 0
    old = mb.get_wait_limit_ns()
    try:
        mb.set_wait_limit_ns(1)
        mb.adapters(X, A, B, Y, idx, rows, src, 128, base=base, status=st)
        torch.cuda.synchronize()
    finally:
        mb.set_wait_limit_ns(old)
    assert st.item() == 5
    st.zero_()
    mb.adapters(X, A, B, Y, idx, rows, src, 128, base=base, status=st)
    assert st.item() == 0 and torch.equal(Y, want)


def map_with_holes(ids, E, align, lead, every, more, device):
    """A map of a program's own: an adapter's rows begin `lead` rows behind its aligned
    start, with a row left empty after every `every` tokens (never the first of 16), and
    `more` empty rows at the end."""
    rows, row = np.full(len(ids), -1), 0
    for e in range(E):
        at = np.nonzero(ids == e)[0]
        place = row + lead
        for i, t in enumerate(at):
            rows[t] = place
            place += 2 if i % every == every - 1 and (place + 1) % 16 else 1
        row = (place + align - 1) // align * align if len(at) else row
    src = np.full(row + more, -1)
    src[rows[rows >= 0]] = np.nonzero(rows >= 0)[0]
    return ou.i32(ids.reshape(-1, 1), device), ou.i32(rows.reshape(-1, 1), device), ou.i32(src, device)


HOLES = [  # tokens, adapters, rank, align, first row, tokens between empty rows, empty rows at the end
    (40, 3, 16, 16, 0, 5, 0), (40, 3, 16, 32, 16, 7, 4000), (300, 4, 64, 64, 48, 100, 20000), (5, 2, 128, 16, 0, 1, 1001),
    (3300, 3, 16, 128, 16, 1000, 0), (3300, 2, 64, 128, 112, 50, 640), (4000, 5, 8, 256, 144, 4, 0),
    (700, 2, 128, 128, 32, 12, 0)]


@pytest.mark.parametrize("T,E,r,align,lead,every,more", HOLES)
def test_adapters_of_a_map_with_empty_rows(T, E, r, align, lead, every, more, cuda):
    """Every token of the map has its result, wherever among the rows of its adapter's
    alignment the tokens begin."""
    rng = np.random.default_rng(T + r)
    K, N = 136, 264
    ids = rng.integers(-1, E, size=T)
    X, base = bf16(rng, (T, K), 1.0, cuda), bf16(rng, (T, N), 1.0, cuda)
    A, B = bf16(rng, (E, r, K), K ** -0.5, cuda), bf16(rng, (E, N, r), r ** -0.5, cuda)
    idx, rows, src = map_with_holes(ids, E, align, lead, every, more, cuda)
    y, size = want64(X, A, B, base, ids.tolist(), None)
    st = ou.status_word(cuda)
    for given in (base, None):
        Y = torch.full((T, N), -77.0, dtype=BF16, device=cuda) if given is not None else base.clone()
        mb.adapters(X, A, B, Y, idx, rows, src, align, base=given, status=st)
        check(Y, y, size)
    assert st.item() == 0


@pytest.mark.parametrize("T,r,align,more", [(40, 16, 16, 0), (40, 16, 16, 4000), (3300, 16, 128, 0)])
def test_adapters_skip_a_bad_first_row_alone(T, r, align, more, cuda):
    """A tile's first row that names no token is reported and skipped; the rows behind
    it keep their results."""
    rng = np.random.default_rng(T + more)
    E, K, N = 2, 320, 264
    ids = np.sort(rng.integers(0, E, size=T))
    X, base = bf16(rng, (T, K), 1.0, cuda), bf16(rng, (T, N), 1.0, cuda)
    A, B = bf16(rng, (E, r, K), K ** -0.5, cuda), bf16(rng, (E, N, r), r ** -0.5, cuda)
    idx, rows, src = map_with_holes(ids, E, align, 0, T, more, cuda)
    y, size = want64(X, A, B, base, ids.tolist(), None)
    lost = src[0].item()
    src[0] = T + 5
    st = ou.status_word(cuda)
    Y = torch.full((T, N), -77.0, dtype=BF16, device=cuda)
    mb.adapters(X, A, B, Y, idx, rows, src, align, base=base, status=st)
    assert st.item() == 6 and (Y[lost] == -77).all()
    keep = torch.arange(T, device=cuda) != lost
    check(Y[keep], y[keep], size[keep])


@pytest.mark.parametrize("T,align", [(40, 16), (3300, 128)])
def test_adapters_of_columns_of_one_buffer(T, align, cuda):
    """X, base and Y as columns of one wider buffer, Y's rows some rows on, and behind
    one another with strides of their own: they share no bytes."""
    rng = np.random.default_rng(T)
    E, r, K, N = 3, 16, 136, 72
    ids = rng.integers(-1, E, size=T)
    A, B = bf16(rng, (E, r, K), K ** -0.5, cuda), bf16(rng, (E, N, r), r ** -0.5, cuda)
    idx, rows, src = slot_map(ids, E, align, cuda)
    for lead in (0, 3):
        for order in ((0, K, K + N), (2 * N, N, 0), (N, 0, N + K)):
            whole = bf16(rng, (T + lead, K + 2 * N), 1.0, cuda)
            X, base = whole[:T, order[0]:order[0] + K], whole[:T, order[1]:order[1] + N]
            Y = whole[lead:, order[2]:order[2] + N]
            y, size = want64(X, A, B, base, ids.tolist(), None)
            mb.adapters(X, A, B, Y, idx, rows, src, align, base=base)
            check(Y, y, size)
    flat = bf16(rng, (1, T * (K + N + 8 + N)), 1.0, cuda)[0]
    X, base = flat[:T * K].view(T, K), flat[T * K:T * (K + N + 8)].view(T, N + 8)[:, :N]
    Y = flat[T * (K + N + 8):].view(T, N)
    y, size = want64(X, A, B, base, ids.tolist(), None)
    mb.adapters(X, A, B, Y, idx, rows, src, align, base=base)
    check(Y, y, size)


@pytest.mark.parametrize("align", [16, 128])
def test_adapters_of_a_mixed_step(align, cuda):
    """Prompts of a few adapters and single tokens of many others, some without one, in
    one call: each token as in a call of its own kind."""
    rng = np.random.default_rng(align)
    E, r, K, N = 40, 32, 640, 1032
    prompts = np.repeat(rng.integers(-1, 3, size=6), [1500, 7, 260, 1, 1033, 399])
    ids = np.concatenate([prompts, rng.permutation(E)[:30], np.full(5, -1)])[rng.permutation(3235)]
    T = len(ids)
    X, base = bf16(rng, (T, K), 1.0, cuda), bf16(rng, (T, N), 1.0, cuda)
    A, B = bf16(rng, (E, r, K), K ** -0.5, cuda), bf16(rng, (E, N, r), r ** -0.5, cuda)
    scale = ou.f32(rng.normal(size=E), cuda)
    idx, rows, src = slot_map(ids, E, align, cuda)
    y, size = want64(X, A, B, base, ids.tolist(), scale)
    st = ou.status_word(cuda)
    Y, Z = torch.full((T, N), -77.0, dtype=BF16, device=cuda), base.clone()
    mb.adapters(X, A, B, Y, idx, rows, src, align, base=base, scale=scale, status=st)
    mb.adapters(X, A, B, Z, idx, rows, src, align, scale=scale, status=st)
    check(Y, y, size)
    assert st.item() == 0 and torch.equal(Y, Z)


@pytest.mark.parametrize("T,E,r,K,N", [(700, 2, 120, 8, 1032), (1400, 2, 64, 320, 264), (700, 3, 128, 72, 8)])
def test_adapters_of_short_prompts_of_a_high_rank(T, E, r, K, N, cuda):
    """In tiles of 128 rows; and with a row that names no token."""
    rng = np.random.default_rng(T + r)
    ids = np.sort(rng.integers(-1, E, size=T))
    X, base = bf16(rng, (T, K), 1.0, cuda), bf16(rng, (T, N), 1.0, cuda)
    A, B = bf16(rng, (E, r, K), K ** -0.5, cuda), bf16(rng, (E, N, r), r ** -0.5, cuda)
    idx, rows, src = slot_map(ids, E, 128, cuda)
    y, size = want64(X, A, B, base, ids.tolist(), None)
    Y, st = torch.full((T, N), -77.0, dtype=BF16, device=cuda), ou.status_word(cuda)
    mb.adapters(X, A, B, Y, idx, rows, src, 128, base=base, status=st)
    check(Y, y, size)
    assert st.item() == 0
    lost = src[33].item()
    src[33] = T + 5
    Y.fill_(-77.0)
    mb.adapters(X, A, B, Y, idx, rows, src, 128, base=base, status=st)
    assert st.item() == 6 and (Y[lost] == -77).all()
    keep = torch.arange(T, device=cuda) != lost
    check(Y[keep], y[keep], size[keep])
