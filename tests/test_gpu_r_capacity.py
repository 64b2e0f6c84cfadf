"""Training steps whose layout is too small: experts that do not fit lose their
choices, which keep their experts and weights but get no row.  Their gradient is
zero, step after step with the same buffers, eager and from a CUDA graph."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_side_gb300 import binding as mb
from oracle import ops as oo
from tests import ops_util as ou

pytestmark = pytest.mark.gpu

T, k, E, N, CAP = 64, 3, 8, 256, 120


def test_choices_without_a_row_have_no_gradient(cuda):
    rng = np.random.default_rng(5)
    logits = torch.empty((T, E), device=cuda)
    idx, w = torch.empty((T, k), dtype=torch.int32, device=cuda), torch.empty((T, k), device=cuda)
    rows, counts = torch.empty_like(idx), torch.empty(E, dtype=torch.int32, device=cuda)
    src = torch.empty(CAP, dtype=torch.int32, device=cuda)
    HC, SHC = torch.empty((CAP, N), dtype=torch.uint8, device=cuda), torch.empty((CAP, 2), dtype=torch.uint8,
                                                                                 device=cuda)
    dY = torch.empty((CAP, N // 2), dtype=torch.bfloat16, device=cuda)
    dH = torch.empty((CAP, N), dtype=torch.bfloat16, device=cuda)
    dw, dl = torch.full((T, k), 1e6, device=cuda), torch.empty((T, E), device=cuda)
    st = ou.status_word(cuda)

    def step():
        mb.route(logits, idx, w, score="sigmoid", renorm=True, status=st)
        mb.slots_contiguous(idx, rows, counts, 1, CAP, src=src, status=st)
        dw.zero_()                       # choices without a row keep what dw held
        mb.swiglu_backward(dY, HC, SHC, dH, w=w, src=src, dw=dw, status=st)
        mb.route_backward(logits, idx, dw, dl, score="sigmoid", renorm=True, status=st)

    def new_inputs():
        logits.copy_(ou.f32(rng.permuted(np.tile(np.linspace(-2, 2, E), (T, 1)), axis=1), cuda))
        q, s = oo.quantize(ou.random_bf16(rng, (CAP, N), 2.0)[1])
        HC.copy_(torch.from_numpy(q))
        SHC.copy_(torch.from_numpy(s))
        d, dv = ou.random_bf16(rng, (CAP, N // 2))
        dY.copy_(d)
        return oo.dequantize(q, s), dv

    def check(h, dv):
        assert st.item() == 4                                       # MG_ERR_CAPACITY
        x, at, r = ou.np64(logits), idx.cpu().numpy(), rows.cpu().numpy()
        gone = r < 0
        assert (at >= 0).all() and gone.any() and not gone.all()
        want = np.zeros((T, k))
        _, _, row_dw = oo.swiglu_backward(dv, h, np.ones(CAP))
        want[~gone] = row_dw[r[~gone]]
        got = ou.np64(dw)
        assert (got[gone] == 0).all()
        # 128 terms, each off by the fast SiLU's error at |g| < 16 and a rounding
        size = np.abs(dv * oo.swiglu(h)).sum(1)
        assert (np.abs(got - want)[~gone] <= (2 * (8 + 1.2 * 16) * 2.0 ** -23 + 128 * ou.U32) * size[r[~gone]]).all()
        ref = oo.route_backward(x, at, got, "sigmoid", True, 1.0)
        big = np.abs(got).max(1, keepdims=True)
        assert (np.abs(ou.np64(dl) - ref) <= 64 * k * ou.U32 * big).all()

    for _ in range(2):
        made = new_inputs()
        st.zero_()
        step()
        check(*made)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        made = new_inputs()
        st.zero_()
        dw.fill_(1e6)
        graph.replay()
        check(*made)
