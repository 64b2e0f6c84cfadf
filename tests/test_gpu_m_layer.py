"""The operators together: the example layer's training step against a float64
evaluation that uses the same 8-bit rows, and its decode step against float64
on the dequantised operands, eager and from a CUDA graph."""
import numpy as np
import pytest
import torch

from examples.moe_layer import MoeLayer
from moe_grouped_gemm_side_gb300 import workloads as wl
from oracle import numerics as on
from oracle import ops as oo
from tests import ops_util as ou

pytestmark = pytest.mark.gpu


def fro(a, b):
    return np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-300)


@pytest.mark.parametrize("T,E,k,dim,inner", [(150, 8, 2, 256, 256), (1, 4, 3, 128, 128), (333, 16, 4, 384, 256)])
def test_training_step(T, E, k, dim, inner, cuda):
    layer = MoeLayer(E, k, dim, inner, groups=2, top_groups=2, scale=1.5, seed=5, device=cuda)
    x = wl.normal_bf16((T, dim), 21, cuda)
    dout = wl.normal_bf16((T, dim), 22, cuda)
    out, s = layer.forward(x)
    g = layer.backward(dout, s)
    assert layer.status.item() == 0
    xv, dv = ou.bf16_np(x), ou.bf16_np(dout)
    W1, W2, R = ou.bf16_np(layer.W1), ou.bf16_np(layer.W2), ou.np64(layer.router)
    idx, w, rows = s["idx"].cpu().numpy(), ou.np64(s["w"]), s["rows"].cpu().numpy()
    # every token has k distinct experts; their weights are the router's
    assert all(len(set(r)) == k and min(r) >= 0 for r in idx.tolist())
    ref_w = oo.route_weights(ou.np64(s["logits"]), idx, "sigmoid", True, 1.5)
    assert np.abs(w - ref_w).max() < 1e-5
    want, dW1, dW2 = np.zeros((T, dim)), np.zeros_like(W1), np.zeros_like(W2)
    dx, dw = np.zeros((T, dim)), np.zeros((T, k))
    hq, hs = s["hq"].cpu().numpy(), s["hs"].cpu().numpy()
    xback = oo.dequantize(s["xq"].cpu().numpy(), s["xs"].cpu().numpy())
    for t in range(T):
        for j in range(k):
            e, r = idx[t, j], rows[t, j]
            h = (W1[e] @ xv[t])[None]
            kept = oo.dequantize(hq[r:r + 1], hs[r:r + 1])
            assert fro(kept, h) < 0.05                        # the 8-bit copy of GEMM1's row
            want[t] += w[t, j] * (W2[e] @ oo.swiglu(h)[0])
            dh, y, d = oo.swiglu_backward((W2[e].T @ dv[t])[None], kept, w[t, j:j + 1])
            dw[t, j] = d[0]
            dW2[e] += np.outer(dv[t], y[0])
            dW1[e] += np.outer(dh[0], xback[t])
            dx[t] += W1[e].T @ dh[0]
    dlogits = oo.route_backward(ou.np64(s["logits"]), idx, dw, "sigmoid", True, 1.5)
    dx += dlogits @ R
    # bf16 at each of the steps between (rows, activations, gradients of rows):
    # a few units of 2^-9 on average
    assert fro(ou.bf16_np(out), want) < 1e-2
    assert fro(ou.np64(g["dW1"]), dW1) < 1e-2 and fro(ou.np64(g["dW2"]), dW2) < 1e-2
    assert fro(ou.np64(g["dx"]), dx) < 1e-2
    assert fro(ou.np64(g["drouter"]), dlogits.T @ xv) < 2e-2


def test_decode_step_and_graph(cuda):
    T, E, k, dim, inner = 23, 8, 2, 256, 384
    layer = MoeLayer(E, k, dim, inner, groups=1, top_groups=1, scale=1.0, seed=9, device=cuda)
    layer.quantise()
    b = layer.decode_buffers(T, 32)
    x = wl.normal_bf16((T, dim), 31, cuda)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.decode(x, b)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            layer.decode(x, b)
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    Q1 = [on.dequant_weight(layer.Q1[e].cpu().numpy(), layer.S1[e].cpu().numpy()) for e in range(E)]
    Q2 = [on.dequant_weight(layer.Q2[e].cpu().numpy(), layer.S2[e].cpu().numpy()) for e in range(E)]
    for seed in (31, 32):
        x.copy_(wl.normal_bf16((T, dim), seed, cuda))
        graph.replay()
        torch.cuda.synchronize()
        assert layer.status.item() == 0
        got = ou.bf16_np(b["out"])
        idx, w = b["idx"].cpu().numpy(), ou.np64(b["w"])
        q, sf = oo.quantize(ou.bf16_np(x))
        xq = oo.dequantize(q, sf)
        want = np.zeros((T, dim))
        for t in range(T):
            for j in range(k):
                y = oo.swiglu((Q1[idx[t, j]] @ xq[t])[None])
                yq, ys = oo.quantize(y)
                want[t] += w[t, j] * (Q2[idx[t, j]] @ oo.dequantize(yq, ys)[0])
        # a code that rounds the other way moves y by 2^-4 of itself; few do
        assert fro(got, want) < 1e-2
        assert torch.equal(b["out"], layer.decode(x, b))
