"""One mixture-of-experts layer on the library's calls: a training step and a
decode step.

Training keeps, per token, an 8-bit copy of its input, and per expert row the
8-bit copy of GEMM1's output; the backward pass rebuilds everything else from
those.  Every call is stream-ordered and reads the routing result on the GPU
only, so nothing here waits for the GPU between the router and the gradients.

    python examples/moe_layer.py            # both steps, timed
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_grouped_gemm_side_gb300 import binding as mb  # noqa: E402
from moe_grouped_gemm_side_gb300 import workloads as wl  # noqa: E402

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class MoeLayer:
    """E experts of hidden size `dim` and inner size `inner` (multiples of 128),
    k experts per token chosen by a sigmoid router with a balance bias.
    W1 [E, 2 inner, dim] holds gate and up rows interleaved in blocks of 128;
    W2 is [E, dim, inner]."""

    def __init__(self, E, k, dim, inner, groups=1, top_groups=1, scale=1.0, seed=0, device="cuda"):
        self.E, self.k, self.dim, self.inner, self.device = E, k, dim, inner, device
        self.routing = dict(score="sigmoid", groups=groups, top_groups=top_groups, group_top=2 if E // groups > 1 else 1,
                            renorm=True, scale=scale)
        self.router = wl.normal_f32((E, dim), seed, device, dim ** -0.5)
        self.bias = torch.zeros(E, device=device)
        self.W1 = wl.normal_bf16((E, 2 * inner, dim), seed + 1, device, dim ** -0.5)
        self.W2 = wl.normal_bf16((E, dim, inner), seed + 2, device, inner ** -0.5)
        self.status = torch.zeros(1, dtype=I32, device=device)

    def _empty(self, *shape, dtype=BF16):
        return torch.empty(shape, dtype=dtype, device=self.device)

    def _route(self, x):
        T = x.shape[0]
        logits = x.float() @ self.router.t()
        idx, w = self._empty(T, self.k, dtype=I32), self._empty(T, self.k, dtype=F32)
        mb.route(logits, idx, w, bias=self.bias, status=self.status, **self.routing)
        return logits, idx, w

    # ------------------------------------------------------------- training
    def forward(self, x):
        """out [T, dim] of bf16 tokens x, and what the backward pass needs."""
        T, st, rows_cap = x.shape[0], self.status, x.shape[0] * self.k
        logits, idx, w = self._route(x)
        rows, counts = self._empty(T, self.k, dtype=I32), self._empty(self.E, dtype=I32)
        src = self._empty(rows_cap, dtype=I32)
        work = self._empty(mb.slots_work_bytes(T * self.k, self.E), dtype=U8)
        # packed segments (align 1) are what the weight gradient reads too
        mb.slots_contiguous(idx, rows, counts, 1, rows_cap, src=src, work=work, status=st)
        A = self._empty(rows_cap, self.dim)
        xq, xs = self._empty(T, self.dim, dtype=U8), self._empty(T, self.dim // 128, dtype=U8)
        mb.dispatch(x, rows, A, CX=xq, SCX=xs, status=st)
        H = self._empty(rows_cap, 2 * self.inner)
        mb.mgemm_contiguous(A, self.W1, H, counts, 1, status=st)
        Y = self._empty(rows_cap, self.inner)
        hq, hs = self._empty(rows_cap, 2 * self.inner, dtype=U8), self._empty(rows_cap, self.inner // 64, dtype=U8)
        mb.swiglu_save(H, Y, hq, hs, src=src)
        D = self._empty(rows_cap, self.dim)
        mb.mgemm_contiguous(Y, self.W2, D, counts, 1, status=st)
        out = self._empty(T, self.dim)
        mb.combine(D, rows, out, w=w, status=st)
        return out, dict(x=x, logits=logits, idx=idx, w=w, rows=rows, counts=counts, src=src, xq=xq, xs=xs, hq=hq, hs=hs)

    def backward(self, dout, saved):
        """Gradients dx, dW1, dW2 and of the router, from dout [T, dim] bf16.
        The transposed weights are laid out here; a program that steps its
        optimizer would lay them out there, once a step."""
        s, st, rows_cap = saved, self.status, saved["src"].numel()
        rows, counts = s["rows"], s["counts"]
        W1t, W2t = self.W1.transpose(1, 2).contiguous(), self.W2.transpose(1, 2).contiguous()
        G = self._empty(rows_cap, self.dim)                     # dout at every expert row
        mb.dispatch(dout, rows, G, status=st)
        dY = self._empty(rows_cap, self.inner)                  # before the routing weight
        mb.mgemm_contiguous(G, W2t, dY, counts, 1, status=st)
        dH, Y = self._empty(rows_cap, 2 * self.inner), self._empty(rows_cap, self.inner)
        dw = torch.zeros_like(s["w"])                           # choices without a row stay 0
        mb.swiglu_backward(dY, s["hq"], s["hs"], dH, w=s["w"], src=s["src"], Y=Y, dw=dw, status=st)
        dW2 = self._empty(self.E, self.dim, self.inner, dtype=F32)
        mb.kgemm_grouped(G, Y, dW2, counts, status=st)
        A = G                                                   # its last reader is done
        mb.dispatch(s["xq"], rows, A, SX=s["xs"], status=st)
        dW1 = self._empty(self.E, 2 * self.inner, self.dim, dtype=F32)
        mb.kgemm_grouped(dH, A, dW1, counts, status=st)
        dA = self._empty(rows_cap, self.dim)
        mb.mgemm_contiguous(dH, W1t, dA, counts, 1, status=st)
        dx = self._empty(dout.shape[0], self.dim, dtype=F32)
        mb.combine(dA, rows, dx, status=st)
        dlogits = torch.empty_like(s["logits"])
        mb.route_backward(s["logits"], s["idx"], dw, dlogits, score=self.routing["score"], renorm=True,
                          scale=self.routing["scale"], status=st)
        dx += dlogits @ self.router
        return dict(dx=dx, dW1=dW1, dW2=dW2, drouter=dlogits.t() @ s["x"].float())

    # --------------------------------------------------------------- decode
    def quantise(self):
        """E4M3 copies of the expert weights for the decode step."""
        pairs1 = [wl.quantize_weight_fp8(self.W1[e].float()) for e in range(self.E)]
        pairs2 = [wl.quantize_weight_fp8(self.W2[e].float()) for e in range(self.E)]
        self.Q1, self.S1 = (torch.stack(t) for t in zip(*pairs1))
        self.Q2, self.S2 = (torch.stack(t) for t in zip(*pairs2))

    def decode_buffers(self, T, M_max):
        """Buffers of a decode step of T tokens, at most M_max rows per expert."""
        E, k, dim, inner = self.E, self.k, self.dim, self.inner
        return dict(M=M_max, idx=self._empty(T, k, dtype=I32), w=self._empty(T, k, dtype=F32),
                    rows=self._empty(T, k, dtype=I32), counts=self._empty(E, dtype=I32),
                    A=self._empty(E, M_max, dim, dtype=U8), SFA=self._empty(E, dim // 128, M_max, dtype=U8),
                    Y=self._empty(E, M_max, inner, dtype=U8), SFY=self._empty(E, inner // 128, M_max, dtype=U8),
                    D=self._empty(E, M_max, dim), out=self._empty(T, dim),
                    work=self._empty(mb.slots_work_bytes(T * k, E), dtype=U8))

    def decode(self, x, b):
        """One decode step in FP8 into the buffers b (can be captured in a CUDA graph)."""
        st = self.status
        logits = x.float() @ self.router.t()
        mb.route(logits, b["idx"], b["w"], bias=self.bias, status=st, **self.routing)
        mb.slots_masked(b["idx"], b["rows"], b["counts"], b["M"], work=b["work"], status=st)
        mb.dispatch(x, b["rows"], b["A"], SFA=b["SFA"], status=st)
        mb.mgemm_masked_swiglu(b["A"], self.Q1, b["Y"], b["counts"], SFA=b["SFA"], SFB=self.S1, SFY=b["SFY"], status=st)
        mb.mgemm_masked(b["Y"], self.Q2, b["D"], b["counts"], SFA=b["SFY"], SFB=self.S2, status=st)
        mb.combine(b["D"], b["rows"], b["out"], w=b["w"], status=st)
        return b["out"]


def _ms(f, reps=10):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    for _ in range(reps):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / reps


def main():
    layer = MoeLayer(E=32, k=8, dim=2048, inner=2048, groups=4, top_groups=2, scale=2.5)
    x = wl.normal_bf16((8192, layer.dim), 11, layer.device)
    dout = wl.normal_bf16((8192, layer.dim), 12, layer.device)
    kept = {}

    def forward():
        kept["out"], kept["saved"] = layer.forward(x)

    print("training, 8192 tokens, 32 experts of 2048 x 2048: forward %.2f ms, backward %.2f ms" % (
        _ms(forward), _ms(lambda: layer.backward(dout, kept["saved"]))))
    layer.quantise()
    tokens = wl.normal_bf16((64, layer.dim), 13, layer.device)
    buffers = layer.decode_buffers(64, 64)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.decode(tokens, buffers)
        graph = torch.cuda.CUDAGraph()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            layer.decode(tokens, buffers)
    torch.cuda.current_stream().wait_stream(stream)
    print("decode, 64 tokens: %.3f ms a call, %.3f ms from a graph" % (
        _ms(lambda: layer.decode(tokens, buffers)), _ms(graph.replay)))
    assert layer.status.item() == 0, mb.status_str(layer.status.item())


if __name__ == "__main__":
    main()
