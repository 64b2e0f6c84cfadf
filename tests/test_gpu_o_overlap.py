"""Slot map and dispatch one after another, over and over into the same buffers:
every dispatch follows the map written just before it, on however many blocks
the two overlap."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_side_gb300 import binding as mb
from oracle import ops as oo
from tests import ops_util as ou

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("src", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,k,E,K", [(61, 4, 16, 512), (900, 8, 40, 256), (9000, 8, 64, 128)])
def test_dispatch_follows_its_map(T, k, E, K, src, cuda):
    rng = np.random.default_rng(T + k)
    steps, cap = 6, T * k + E * 16
    maps = [ou.random_choices(rng, T, k, E) for _ in range(steps)]
    idx = [ou.i32(m, cuda) for m in maps]
    x = [torch.from_numpy(rng.integers(0, 119, size=(T, K)).astype(np.uint8)).to(cuda) for _ in range(steps)]
    sx = [torch.from_numpy(rng.integers(120, 134, size=(T, K // 128)).astype(np.uint8)).to(cuda) for _ in range(steps)]
    if src == "bf16":
        x = [v.view(torch.float8_e4m3fn).to(torch.bfloat16) for v in x]
    rows, counts = torch.empty((T, k), dtype=torch.int32, device=cuda), torch.empty(E, dtype=torch.int32, device=cuda)
    work = torch.empty(mb.slots_work_bytes(T * k, E), dtype=torch.uint8, device=cuda)
    X, SX = torch.empty_like(x[0]), torch.empty_like(sx[0])
    A = [torch.zeros((cap, K), dtype=torch.bfloat16, device=cuda) for _ in range(4 * steps)]
    got = []
    for i in range(4 * steps):                       # nothing waits for the GPU in here
        X.copy_(x[i % steps])
        SX.copy_(sx[i % steps])
        mb.slots_contiguous(idx[i % steps], rows, counts, 16, cap, work=work)
        mb.dispatch(X, rows, A[i], SX=SX if src == "e4m3" else None)
        got.append(rows.clone())
    torch.cuda.synchronize()
    for i in range(4 * steps):
        want, _, _, _ = oo.slots(maps[i % steps], E, align_q=16, rows_cap=cap)
        assert np.array_equal(got[i].cpu().numpy(), want)
        at = torch.from_numpy(np.argwhere(want >= 0)).to(cuda)
        v = x[i % steps]
        if src == "e4m3":
            scale = torch.exp2(sx[i % steps].float() - 127).repeat_interleave(128, 1)
            v = (v.view(torch.float8_e4m3fn).float() * scale).to(torch.bfloat16)
        r = got[i][at[:, 0], at[:, 1]].long()
        expect = torch.zeros_like(A[i])
        expect[r] = v[at[:, 0]]
        assert torch.equal(A[i], expect)
