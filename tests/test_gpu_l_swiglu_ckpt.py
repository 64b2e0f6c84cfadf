"""SwiGLU with its rows kept in 8 bits, and its backward pass from them, on the
GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_side_gb300 import binding as mb
from oracle import ops as oo
from tests import ops_util as ou
from tests.gpu_util import sentinel_like
from tests.test_gpu_k_rows import layout

pytestmark = pytest.mark.gpu

CASES = [(1, 1, 1, 256, "contiguous", 1), (3, 2, 4, 256, "masked", 16), (11, 3, 5, 768, "contiguous", 16),
         (29, 4, 8, 1280, "contiguous", 128), (9, 2, 3, 4096, "masked", 16), (700, 2, 7, 512, "contiguous", 8),
         (13, 2, 4, 2816, "contiguous", 16), (7, 3, 3, 4352, "contiguous", 8)]


def fast_tol(g):
    """Relative error of SiLU and of 1 / (1 + e^-g) as the kernels compute them."""
    return (8 + 1.2 * np.abs(g)) * 2.0 ** -23


@pytest.mark.parametrize("out", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,k,E,N,kind,align", CASES)
def test_save(T, k, E, N, kind, align, out, cuda):
    rng = np.random.default_rng(T + N)
    _, _, src, lead = layout(rng, T, k, E, kind, align)
    R, G = int(np.prod(lead)), lead[-1]
    H, hv = ou.random_bf16(rng, (R, N), 2.0)
    live = src >= 0
    H[torch.from_numpy(~live)] = float("nan")
    Y = torch.full(lead + (N // 2,), 0x7D, dtype=torch.uint8, device=cuda) if out == "e4m3" else \
        sentinel_like(lead + (N // 2,), cuda)
    SFY = torch.full((R // G, N // 256, G), 0xEE, dtype=torch.uint8, device=cuda) if out == "e4m3" else None
    HC = torch.full((R, N), 0x7D, dtype=torch.uint8, device=cuda)
    SHC = torch.full((R, N // 128), 0xEE, dtype=torch.uint8, device=cuda)
    keep = Y.clone()
    mb.swiglu_save(H.view(lead + (N,)).to(cuda), Y, HC, SHC, SFY=SFY, src=ou.i32(src, cuda))
    q, s = oo.quantize(hv[live])
    hc, shc = HC.cpu().numpy(), SHC.cpu().numpy()
    assert np.array_equal(hc[live], q) and np.array_equal(shc[live], s)
    assert (hc[~live] == 0x7D).all() and (shc[~live] == 0xEE).all()
    ref = oo.swiglu(hv[live])
    g, _ = oo.gate_up(hv[live])
    Y2, K2 = Y.view(R, -1).cpu(), keep.view(R, -1).cpu()
    dead = torch.from_numpy(~live)
    assert torch.equal(Y2[dead].view(torch.uint8), K2[dead].view(torch.uint8))
    if out == "bf16":
        err = np.abs(ou.bf16_np(Y2[~dead]) - ref)
        assert (err <= (ou.BF16 + 2 * fast_tol(g)) * np.abs(ref)).all()
        return
    sf = SFY.cpu().numpy()
    r = np.nonzero(live)[0]
    got_s = sf[r // G, :, r % G]
    assert (sf.transpose(0, 2, 1).reshape(R, -1)[~live] == 0xEE).all()
    y = oo.dequantize(Y2[~dead].numpy(), got_s)
    # the block's scale may sit one step off only where its maximum is within
    # the fast SiLU's error of the step; a code is within half a step of y
    amax = np.abs(ref).reshape(len(r), -1, 128).max(2)
    step = np.exp2(got_s.astype(np.float64) - 127)
    assert (amax <= 448 * step * (1 + 1e-4)).all() and (amax >= 224 * step * (1 - 1e-4)).all()
    quantum = np.repeat(step, 128, 1) * np.exp2(np.maximum(np.floor(np.log2(
        np.maximum(np.abs(ref) / np.repeat(step, 128, 1), 2.0 ** -20))), -6) - 3)
    assert (np.abs(y - ref) <= quantum * (0.5 + 1e-3) + 2 * fast_tol(g) * np.abs(ref)).all()


@pytest.mark.parametrize("T,k,E,N,kind,align", CASES)
@pytest.mark.parametrize("full", [True, False])
def test_backward(T, k, E, N, kind, align, full, cuda):
    rng = np.random.default_rng(2 * T + N)
    rows, _, src, lead = layout(rng, T, k, E, kind, align)
    R = int(np.prod(lead))
    live = src >= 0
    _, hv = ou.random_bf16(rng, (R, N), 2.0)
    q, s = oo.quantize(hv)
    h = oo.dequantize(q, s)
    q[~live], s[~live] = 0x7F, 0xFF                          # rows of no choice hold NaN
    dY, dv = ou.random_bf16(rng, (R, N // 2))
    dY[torch.from_numpy(~live)] = float("nan")
    w = rng.normal(size=(T, k)).astype(np.float32)
    wr = np.ones(R)
    wr[live] = w.reshape(-1)[src[live]]
    if not full:
        wr[:] = 1.0
    dH, Y = sentinel_like(lead + (N,), cuda), sentinel_like(lead + (N // 2,), cuda)
    kH, kY = dH.clone(), Y.clone()
    dw = torch.full((T, k), 9.0, device=cuda)
    st = ou.status_word(cuda)
    more = dict(w=ou.f32(w, cuda), Y=Y, dw=dw) if full else {}
    mb.swiglu_backward(dY.view(lead + (N // 2,)).to(cuda), torch.from_numpy(q).to(cuda),
                       torch.from_numpy(s).to(cuda), dH, src=ou.i32(src, cuda), status=st, **more)
    assert st.item() == 0
    rH, rY, rw = oo.swiglu_backward(dv[live], h[live], wr[live])
    g, u = oo.gate_up(h[live])
    tol = fast_tol(g)
    sig = oo._sigmoid(g)
    d = np.abs(dv[live] * wr[live][:, None])
    # dg = d u sigma (1 + g (1 - sigma)): every term within its own fast-sigmoid
    # error, the sum bounded by its terms' magnitudes
    bg = 4 * tol * d * np.abs(u) * sig * (1 + np.abs(g))
    bu = 4 * tol * d * np.abs(g) * sig
    got = ou.bf16_np(dH.view(R, N))[live]
    assert (np.abs(got - rH) <= (ou.BF16 + 4 * ou.U32) * np.abs(rH) + oo.interleave(bg, bu)).all()
    dead = torch.from_numpy(~live).to(cuda)
    assert torch.equal(dH.view(R, N)[dead].view(torch.int16), kH.view(R, N)[dead].view(torch.int16))
    if not full:
        return
    gy = ou.bf16_np(Y.view(R, -1))[live]
    assert (np.abs(gy - rY) <= (ou.BF16 + 4 * tol) * np.abs(rY) + 1e-38).all()
    assert torch.equal(Y.view(R, -1)[dead].view(torch.int16), kY.view(R, -1)[dead].view(torch.int16))
    y = oo.swiglu(h[live])
    mag = np.abs(dv[live] * y).sum(1)
    bound = (N // 2) * ou.U32 * mag + (2 * tol * np.abs(dv[live] * y)).sum(1)
    gw = ou.np64(dw).reshape(-1)
    assert (np.abs(gw[src[live]] - rw) <= bound + 1e-38).all()
    gone = np.setdiff1d(np.arange(T * k), src[live])
    assert (gw[gone] == 9.0).all()


def test_all_rows_without_a_map(cuda):
    rng = np.random.default_rng(3)
    R, N = 37, 512
    H, hv = ou.random_bf16(rng, (R, N))
    Y = torch.empty((R, N // 2), dtype=torch.bfloat16, device=cuda)
    HC, SHC = torch.empty((R, N), dtype=torch.uint8, device=cuda), torch.empty((R, 4), dtype=torch.uint8, device=cuda)
    mb.swiglu_save(H.to(cuda), Y, HC, SHC)
    q, s = oo.quantize(hv)
    assert np.array_equal(HC.cpu().numpy(), q) and np.array_equal(SHC.cpu().numpy(), s)
    dY, dv = ou.random_bf16(rng, (R, N // 2))
    dH = torch.empty((R, N), dtype=torch.bfloat16, device=cuda)
    mb.swiglu_backward(dY.to(cuda), HC, SHC, dH)
    rH, _, _ = oo.swiglu_backward(dv, oo.dequantize(q, s), np.ones(R))
    assert np.abs(ou.bf16_np(dH) - rH).max() <= (ou.BF16 + 2.0 ** -18) * np.abs(rH).max()


def test_large_gates(cuda):
    """SiLU's tails: far below zero everything vanishes, far above SiLU is g and
    its slope 1; no NaN comes out of finite rows."""
    N = 256
    g = torch.tensor([-300.0, -100.0, -88.0, -20.0, 0.0, 20.0, 88.0, 100.0, 300.0] + [1.0] * 119)
    h = torch.cat([g, torch.full((128,), 2.0)])[None].to(torch.bfloat16)
    Y = torch.empty((1, 128), dtype=torch.bfloat16, device=cuda)
    HC, SHC = torch.empty((1, N), dtype=torch.uint8, device=cuda), torch.empty((1, 2), dtype=torch.uint8, device=cuda)
    mb.swiglu_save(h.to(cuda), Y, HC, SHC)
    assert torch.isfinite(Y.float()).all() and (Y[0, :2].abs() < 1e-30).all() and Y[0, 8] == 600
    dH = torch.empty((1, N), dtype=torch.bfloat16, device=cuda)
    mb.swiglu_backward(torch.ones((1, 128), dtype=torch.bfloat16, device=cuda), HC, SHC, dH)
    assert torch.isfinite(dH.float()).all()
    assert (dH[0, :2].abs() < 1e-30).all() and dH[0, 8] == 2.0 and dH[0, 128 + 4] == 0.0


def test_src_past_the_weights_is_reported(cuda):
    R, N = 3, 256
    HC = torch.zeros((R, N), dtype=torch.uint8, device=cuda)
    SHC = torch.full((R, 2), 127, dtype=torch.uint8, device=cuda)
    dY = torch.ones((R, 128), dtype=torch.bfloat16, device=cuda)
    dH = sentinel_like((R, N), cuda)
    keep = dH.clone()
    st = ou.status_word(cuda)
    mb.swiglu_backward(dY, HC, SHC, dH, w=torch.ones(2, device=cuda), src=ou.i32([0, 2, 1], cuda), status=st)
    assert st.item() == 6 and torch.equal(dH[1].view(torch.int16), keep[1].view(torch.int16))
    assert (dH[[0, 2]] == 0).all()


def test_offsets_past_2_31_elements(cuda):
    R, N = 600000, 4096
    rng = np.random.default_rng(6)
    src = torch.full((R,), -1, dtype=torch.int32, device=cuda)
    src[R - 1] = 0
    H = torch.empty((R, N), dtype=torch.bfloat16, device=cuda)
    h, hv = ou.random_bf16(rng, (1, N))
    H[R - 1] = h[0].to(cuda)
    Y = torch.empty((R, N // 2), dtype=torch.bfloat16, device=cuda)
    HC, SHC = torch.empty((R, N), dtype=torch.uint8, device=cuda), torch.empty((R, N // 128), dtype=torch.uint8,
                                                                               device=cuda)
    mb.swiglu_save(H, Y, HC, SHC, src=src)
    q, s = oo.quantize(hv)
    assert np.array_equal(HC[R - 1].cpu().numpy(), q[0]) and np.array_equal(SHC[R - 1].cpu().numpy(), s[0])
    dY, dv = ou.random_bf16(rng, (1, N // 2))
    Y[R - 1] = dY[0].to(cuda)
    mb.swiglu_backward(Y, HC, SHC, H, src=src)
    rH, _, _ = oo.swiglu_backward(dv, oo.dequantize(q, s), np.ones(1))
    assert np.abs(ou.bf16_np(H[R - 1]) - rH[0]).max() <= (ou.BF16 + 2.0 ** -18) * np.abs(rH).max()


def test_gradient_against_differences(cuda):
    """Central differences in the oracle's forward at the checkpointed rows: the
    kernel's dH is bf16, so 2^-8 of the gradient's size is the finest claim."""
    rng = np.random.default_rng(12)
    _, hv = ou.random_bf16(rng, (2, 256), 1.5)
    q, s = oo.quantize(hv)
    h = oo.dequantize(q, s)
    dY, dv = ou.random_bf16(rng, (2, 128))
    dH = torch.empty((2, 256), dtype=torch.bfloat16, device=cuda)
    mb.swiglu_backward(dY.to(cuda), torch.from_numpy(q).to(cuda), torch.from_numpy(s).to(cuda), dH)
    got, eps = ou.bf16_np(dH), 1e-5
    for c in range(0, 256, 17):
        a, b = h.copy(), h.copy()
        a[:, c] += eps
        b[:, c] -= eps
        diff = ((oo.swiglu(a) - oo.swiglu(b)) * dv).sum(1) / (2 * eps)
        assert (np.abs(diff - got[:, c]) <= 2.0 ** -8 * np.maximum(np.abs(diff), 1e-3)).all()


@pytest.mark.parametrize("N", [256, 1280, 2816])
def test_backward_of_many_rows(N, cuda):
    """Enough rows that few threads share one."""
    rng = np.random.default_rng(N)
    R, n = 9000, 9100
    src = rng.permutation(n)[:R].astype(np.int64)
    src[rng.random(R) < 0.2] = -1
    live = src >= 0
    q = rng.integers(0, 127, size=(R, N)).astype(np.uint8) | (rng.integers(0, 2, size=(R, N)) << 7).astype(np.uint8)
    s = rng.integers(116, 122, size=(R, N // 128)).astype(np.uint8)
    h = oo.dequantize(q, s)
    dY, dv = ou.random_bf16(rng, (R, N // 2))
    w = rng.normal(size=n).astype(np.float32)
    dH, Y = sentinel_like((R, N), cuda), sentinel_like((R, N // 2), cuda)
    dw = torch.full((n,), 9.0, device=cuda)
    mb.swiglu_backward(dY.to(cuda), torch.from_numpy(q).to(cuda), torch.from_numpy(s).to(cuda), dH,
                       w=ou.f32(w, cuda), src=ou.i32(src, cuda), Y=Y, dw=dw)
    rH, rY, rw = oo.swiglu_backward(dv[live], h[live], w[src[live]].astype(np.float64))
    g, u = oo.gate_up(h[live])
    tol, sig = fast_tol(g), oo._sigmoid(g)
    d = np.abs(dv[live] * w[src[live]][:, None])
    bound = oo.interleave(4 * tol * d * np.abs(u) * sig * (1 + np.abs(g)), 4 * tol * d * np.abs(g) * sig)
    assert (np.abs(ou.bf16_np(dH)[live] - rH) <= (ou.BF16 + 4 * ou.U32) * np.abs(rH) + bound + 1e-38).all()
    assert (np.abs(ou.bf16_np(Y)[live] - rY) <= (ou.BF16 + 4 * tol) * np.abs(rY) + 1e-38).all()
    y = oo.swiglu(h[live])
    lim = (N // 2) * ou.U32 * np.abs(dv[live] * y).sum(1) + (2 * tol * np.abs(dv[live] * y)).sum(1)
    got = ou.np64(dw)
    assert (np.abs(got[src[live]] - rw) <= lim + 1e-38).all()
    gone = np.setdiff1d(np.arange(n), src[live])
    assert (got[gone] == 9.0).all()
    dead = torch.from_numpy(~live).to(cuda)
    assert torch.equal(dH[dead].view(torch.int16), sentinel_like((int((~live).sum()), N), cuda).view(torch.int16))


@pytest.mark.parametrize("E,M,filled", [(24, 304, 0.2), (64, 128, 0.05), (3, 4096, 0.5), (160, 16, 0.3)])
def test_runs_of_rows_without_a_choice(E, M, filled, cuda):
    """Buffers whose length divides, or is divided by, any count of blocks: every
    row that holds a choice is done once, the others are left alone."""
    N, R = 512, E * M
    rng = np.random.default_rng(M)
    src = np.full((E, M), -1, dtype=np.int64)
    at = 0
    for e in range(E):
        n = int(rng.integers(0, int(M * filled) * 2 + 2)) if e % 7 else 0
        n = min(n, M)
        src[e, :n] = at + np.arange(n)
        at += n
    src = src.reshape(-1)
    live = src >= 0
    h, hv = ou.random_bf16(rng, (R, N))
    h[torch.from_numpy(~live)] = float("nan")
    st = ou.status_word(cuda)
    Y, HC = sentinel_like((R, N // 2), cuda), torch.full((R, N), 0x5A, dtype=torch.uint8, device=cuda)
    SHC = torch.full((R, N // 128), 0x5A, dtype=torch.uint8, device=cuda)
    keep = Y.clone()
    s_dev = ou.i32(src, cuda)
    mb.swiglu_save(h.to(cuda), Y, HC, SHC, src=s_dev)
    q, s = oo.quantize(hv)
    want_q, want_s = np.full((R, N), 0x5A, np.uint8), np.full((R, N // 128), 0x5A, np.uint8)
    want_q[live], want_s[live] = q[live], s[live]
    assert np.array_equal(HC.cpu().numpy(), want_q) and np.array_equal(SHC.cpu().numpy(), want_s)
    dead = torch.from_numpy(~live).to(cuda)
    assert torch.equal(Y[dead].view(torch.int16), keep[dead].view(torch.int16))
    w = torch.from_numpy(rng.normal(size=at).astype(np.float32))
    dY, dv = ou.random_bf16(rng, (R, N // 2))
    dH, dw = sentinel_like((R, N), cuda), torch.full((at,), 9.0, device=cuda)
    kH = dH.clone()
    mb.swiglu_backward(dY.to(cuda), HC, SHC, dH, w=w.to(cuda), src=s_dev, dw=dw, status=st)
    assert st.item() == 0
    assert torch.equal(dH[dead].view(torch.int16), kH[dead].view(torch.int16))
    hq = oo.dequantize(q, s)[live]
    rH, _, rw = oo.swiglu_backward(dv[live], hq, w.numpy()[src[live]])
    g, u = oo.gate_up(hq)
    tol = fast_tol(g)
    d = np.abs(dv[live] * w.numpy()[src[live]][:, None])
    sig = oo._sigmoid(g)
    bound = oo.interleave(4 * tol * d * np.abs(u) * sig * (1 + np.abs(g)), 4 * tol * d * np.abs(g) * sig)
    assert (np.abs(ou.bf16_np(dH)[live] - rH) <= (ou.BF16 + 4 * ou.U32) * np.abs(rH) + bound).all()
    y = oo.swiglu(hq)
    mag = (N // 2) * ou.U32 * np.abs(dv[live] * y).sum(1) + (2 * tol * np.abs(dv[live] * y)).sum(1)
    assert (np.abs(ou.np64(dw)[src[live]] - rw) <= mag + 1e-38).all()
