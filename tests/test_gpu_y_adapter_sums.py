"""Adapters whose rank sums pass the largest bf16 or fp32, on the GPU against the
formula in float64: an infinite sum gives the infinities of its products, as in the
formula, and a finite one its products.  Tolerances as in the operator's own tests."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_side_gb300 import binding as mb
from tests import ops_util as ou
from tests.test_gpu_u_adapters import BF16, bf16, check, slot_map, want64

pytestmark = pytest.mark.gpu

FORMS = [(40, 8, 16), (40, 128, 16), (300, 64, 64), (3300, 16, 128), (3300, 64, 128)]      # tokens, rank, align


def operands(T, r, align, cuda):
    rng = np.random.default_rng(T + r)
    E, K, N = 2, 136, 264
    ids = np.arange(T) % E
    X = torch.zeros(T, K, dtype=BF16, device=cuda)
    X[:, 2:] = bf16(rng, (T, K - 2), 1.0, cuda)
    A, B = bf16(rng, (E, r, K), K ** -0.5, cuda), bf16(rng, (E, N, r), r ** -0.5, cuda)
    base = bf16(rng, (T, N), 1.0, cuda)
    return ids, X, A, B, base, slot_map(ids, E, align, cuda)


@pytest.mark.parametrize("T,r,align", FORMS)
def test_adapters_with_an_infinite_sum(T, r, align, cuda):
    """The third rank's sum of two tokens is +inf and -inf: their Y are the infinities
    of that rank's column of B, the other tokens' bits do not change."""
    ids, X, A, B, base, (idx, rows, src) = operands(T, r, align, cuda)
    A[:, :, :2] = 0
    A[:, 2, 0] = 1e38
    B[:, :, 2] = torch.where(B[:, :, 2] < 0, -0.25, 0.25).to(BF16)
    clean, Y = torch.empty_like(base), torch.empty_like(base)
    mb.adapters(X, A, B, clean, idx, rows, src, align, base=base)
    up, down = T // 2, T - 1
    X[up, 0], X[down, 0] = 8.0, -8.0
    mb.adapters(X, A, B, Y, idx, rows, src, align, base=base)
    for t, sign in ((up, 1.0), (down, -1.0)):
        assert torch.equal(Y[t].float(), sign * torch.sign(B[ids[t], :, 2].float()) * torch.inf)
    rest = torch.ones(T, dtype=torch.bool, device=cuda)
    rest[up] = rest[down] = False
    assert torch.equal(Y[rest], clean[rest])


@pytest.mark.parametrize("T,r,align", FORMS)
def test_adapters_with_a_sum_past_the_largest_bf16(T, r, align, cuda):
    """A sum of 3.3975e38, which bf16 would round to infinity, times a small B; and of
    both signs."""
    ids, X, A, B, base, (idx, rows, src) = operands(T, r, align, cuda)
    X[:, 2:] = 0                             # the sum is those two terms
    A[:, 2, 0], A[:, 2, 1] = torch.finfo(BF16).max, 8e35
    B[:, :, 2] *= 2.0 ** -100
    X[::3, :2], X[1::3, :2] = 1.0, -1.0
    total = A[0, 2, 0].float() + A[0, 2, 1].float()
    assert total.isfinite() and total.to(BF16).isinf()
    A[:, :2], A[:, 3:] = 0, 0
    y, size = want64(X, A, B, base, ids.tolist(), None)
    Y = torch.empty_like(base)
    mb.adapters(X, A, B, Y, idx, rows, src, align, base=base)
    check(Y, y, size)
