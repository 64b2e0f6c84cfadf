"""Adapters at the edges of what their interface allows, on the GPU.  Tolerances as
in the operator's own tests."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_side_gb300 import binding as mb
from tests import ops_util as ou
from tests.test_gpu_u_adapters import BF16, bf16, slot_map

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
