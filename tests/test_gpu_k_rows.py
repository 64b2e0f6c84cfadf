"""Slot map, dispatch, combine and its gradients on the GPU against the float64
oracle.  Maps, copies, codes and scales are compared bit for bit; rows that a
call must not write hold a sentinel."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_side_gb300 import binding as mb
from oracle import ops as oo
from tests import ops_util as ou
from tests.gpu_util import sentinel_like

pytestmark = pytest.mark.gpu


def run_slots(idx, E, device, align=None, cap=None, M=None, want_src=True):
    T, k = idx.shape
    total = E * M if M is not None else cap
    rows = torch.full((T, k), -9, dtype=torch.int32, device=device)
    counts = torch.full((E,), -9, dtype=torch.int32, device=device)
    src = torch.full((total,), -9, dtype=torch.int32, device=device) if want_src else None
    wb = mb.slots_work_bytes(T * k, E)
    work = torch.full((wb // 4,), 12345, dtype=torch.int32, device=device) if wb else None
    st = ou.status_word(device)
    d = ou.i32(idx, device)
    if M is not None:
        mb.slots_masked(d, rows, counts, M, src=src, work=work, status=st)
    else:
        mb.slots_contiguous(d, rows, counts, align, cap, src=src, work=work, status=st)
    return rows.cpu().numpy(), counts.cpu().numpy(), None if src is None else src.cpu().numpy(), st.item()


SLOT_CASES = [(0, 2, 5), (1, 1, 1), (1, 8, 64), (3, 2, 1), (33, 3, 7), (500, 8, 8), (512, 8, 256), (513, 8, 256),
              (1365, 3, 1024), (1366, 3, 33), (9001, 2, 64), (5000, 7, 160), (7001, 7, 96), (20001, 4, 33)]


@pytest.mark.parametrize("T,k,E", SLOT_CASES)
def test_slots(T, k, E, cuda):
    rng = np.random.default_rng(T * 31 + E)
    idx = ou.random_choices(rng, T, k, E)
    n = T * k
    for align in (1, 16, 128):
        cap = n + E * (align - 1) + 3
        want = oo.slots(idx, E, align_q=align, rows_cap=cap)
        rows, counts, src, st = run_slots(idx, E, cuda, align=align, cap=cap)
        assert st == 0
        assert np.array_equal(rows, want[0]) and np.array_equal(counts, want[1]) and np.array_equal(src, want[2])
    most = int(max((idx == e).sum() for e in range(E))) if n else 0
    for M in (max(most, 1), most // 2 + 1):
        want = oo.slots(idx, E, M_max=M)
        rows, counts, src, st = run_slots(idx, E, cuda, M=M)
        assert (st == 4) == want[3]
        assert np.array_equal(rows, want[0]) and np.array_equal(counts, want[1]) and np.array_equal(src, want[2])


def test_slots_capacity_and_bad_choices(cuda):
    rng = np.random.default_rng(2)
    for T, k, E in ((60, 4, 12), (3000, 3, 40)):
        idx = ou.random_choices(rng, T, k, E)
        for align in (1, 16):
            full = oo.slots(idx, E, align_q=align, rows_cap=T * k + E * align)
            end = int(-(-full[1] // align).sum()) * align
            for cap in (end, end - 1, end // 2, 1):
                want = oo.slots(idx, E, align_q=align, rows_cap=cap)
                rows, counts, src, st = run_slots(idx, E, cuda, align=align, cap=cap)
                assert (st == 4) == want[3], (cap, end)
                assert np.array_equal(rows, want[0]) and np.array_equal(src, want[2])
                assert np.array_equal(counts, want[1])
        bad = idx.copy()
        bad[1, 0], bad[2, 1] = E, -2
        want = oo.slots(bad, E, align_q=16, rows_cap=T * k + E * 16)
        rows, counts, _, st = run_slots(bad, E, cuda, align=16, cap=T * k + E * 16, want_src=False)
        assert st == 6 and np.array_equal(rows, want[0]) and np.array_equal(counts, want[1])


def test_slots_one_hot_expert_and_all_dropped(cuda):
    for n in (4096, 4097, 70000):
        idx = np.zeros((n, 1), dtype=np.int64)
        rows, counts, src, st = run_slots(idx, 3, cuda, align=128, cap=n + 400)
        assert st == 0 and np.array_equal(rows[:, 0], np.arange(n)) and counts.tolist() == [n, 0, 0]
        assert np.array_equal(src[:n], np.arange(n)) and (src[n:] == -1).all()
        rows, counts, src, st = run_slots(idx - 1, 3, cuda, align=128, cap=300)
        assert st == 0 and (rows == -1).all() and counts.tolist() == [0, 0, 0] and (src == -1).all()


def layout(rng, T, k, E, kind, align=16):
    idx = ou.random_choices(rng, T, k, E)
    if kind == "masked":
        M = (max(16, int(max([(idx == e).sum() for e in range(E)]))) + 15) // 16 * 16
        rows, counts, src, _ = oo.slots(idx, E, M_max=M)
        return rows, counts, src, (E, M)
    cap = (T * k + E * (align - 1) + 15) // 16 * 16
    rows, counts, src, _ = oo.slots(idx, E, align_q=align, rows_cap=cap)
    return rows, counts, src, (cap,)


ROW_CASES = [(1, 1, 1, 128, "contiguous", 16), (5, 2, 4, 128, "masked", 16), (13, 3, 7, 384, "contiguous", 16),
             (37, 8, 16, 640, "contiguous", 128), (20, 4, 6, 2176, "masked", 16), (3, 32, 40, 256, "contiguous", 16),
             (9, 2, 5, 7168, "contiguous", 32)]


@pytest.mark.parametrize("src", ["bf16", "e4m3"])
@pytest.mark.parametrize("dst", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,k,E,K,kind,align", ROW_CASES)
def test_dispatch(T, k, E, K, kind, align, src, dst, cuda):
    rng = np.random.default_rng(T + K)
    rows, _, _, lead = layout(rng, T, k, E, kind, align)
    x, xv = ou.random_bf16(rng, (T, K), 3.0)
    x[0, :128] = 0
    xv[0, :128] = 0
    q, s = oo.quantize(xv)
    R = int(np.prod(lead))
    G = lead[-1]
    st = ou.status_word(cuda)
    A = torch.full(lead + (K,), 0x7D, dtype=torch.uint8, device=cuda) if dst == "e4m3" else \
        sentinel_like(lead + (K,), cuda)
    SFA = torch.full((R // G, K // 128, G), 0xEE, dtype=torch.uint8, device=cuda) if dst == "e4m3" else None
    kw = {}
    if src == "bf16":
        X = x.to(cuda)
        kw["CX"] = torch.zeros((T, K), dtype=torch.uint8, device=cuda)
        kw["SCX"] = torch.zeros((T, K // 128), dtype=torch.uint8, device=cuda)
    else:
        X = torch.from_numpy(q).to(cuda)
        kw["SX"] = torch.from_numpy(s).to(cuda)
    before = A.clone()
    mb.dispatch(X, ou.i32(rows, cuda), A, SFA=SFA, status=st, **kw)
    assert st.item() == 0
    if src == "bf16":
        assert np.array_equal(kw["CX"].cpu().numpy(), q) and np.array_equal(kw["SCX"].cpu().numpy(), s)
    A2, B2 = A.view(R, K).cpu(), before.view(R, K).cpu()
    sf = None if SFA is None else SFA.cpu().numpy()
    if dst == "bf16":
        want = x if src == "bf16" else torch.from_numpy(oo.dequantize(q, s)).to(torch.bfloat16)
    filled = set()
    for t in range(T):
        for j in range(k):
            r = int(rows[t, j])
            if r < 0:
                continue
            filled.add(r)
            if dst == "e4m3":
                assert np.array_equal(A2[r].numpy(), q[t])
                assert np.array_equal(sf[r // G, :, r % G], s[t])
            else:
                assert torch.equal(A2[r].view(torch.int16), want[t].view(torch.int16))
    for r in range(R):
        if r not in filled:
            assert torch.equal(A2[r].view(torch.uint8), B2[r].view(torch.uint8))
            if sf is not None:
                assert (sf[r // G, :, r % G] == 0xEE).all()


def test_dispatch_extremes(cuda):
    """Infinities, NaN, the largest and the smallest values survive as the
    checkpoint format says; fp32-range scales at both ends."""
    K = 256
    x = torch.zeros(4, K, dtype=torch.bfloat16)
    big = torch.finfo(torch.bfloat16).max
    x[0, 0], x[0, 1], x[0, 200] = float("inf"), 1.0, -2.0
    x[1, 3], x[1, 4] = float("nan"), 5.0
    x[2, 0], x[2, 1], x[2, 130] = big, -big, 2.0 ** -133
    x[3, 9], x[3, 10] = 448.0, 450.0
    rows = ou.i32([[0], [1], [2], [3]], cuda)
    A = torch.zeros((4, K), dtype=torch.uint8, device=cuda)
    SFA = torch.zeros((1, 2, 4), dtype=torch.uint8, device=cuda)
    mb.dispatch(x.to(cuda), rows, A, SFA=SFA)
    back = torch.zeros((4, K), dtype=torch.bfloat16, device=cuda)
    mb.dispatch(A, rows, back, SX=SFA[0].t().contiguous())
    a, b, sf = A.cpu(), back.cpu(), SFA[0].cpu()
    assert b[0, 0] == float("inf") and b[0, 1] == 0 and abs(b[0, 200] + 2.0) <= 2.0 ** -3
    assert torch.isnan(b[1, 3].float()) and b[1, 4] == 5.0
    # the nearest code of the largest finite values is 256 at 2^120: 2^128, past the type
    assert sf[0, 2] == 247 and a[2, 0] == 0x78 and b[2, 0] == float("inf") and b[2, 1] == float("-inf")
    assert sf[1, 2] == 1 and b[2, 130] == 2.0 ** -133          # code 2^-7 at the smallest scale, 2^-126
    assert sf[0, 3] == 128 and b[3, 9] == 448 and b[3, 10] == 448   # 450 needs the scale 2


@pytest.mark.parametrize("K", [8, 24, 136, 1000, 4096])
def test_bf16_rows_of_any_width(K, cuda):
    """bf16 dispatch and combine take any multiple of eight columns, and token
    rows further apart than K."""
    rng = np.random.default_rng(K)
    T, k, E = 11, 3, 5
    rows, _, _, lead = layout(rng, T, k, E, "contiguous", 1)
    wide, wv = ou.random_bf16(rng, (T, K + 16))
    wide = wide.to(cuda)
    A = sentinel_like(lead + (K,), cuda)
    r = ou.i32(rows, cuda)
    mb.dispatch(wide[:, 8:8 + K], r, A)
    got = A.cpu()
    for t in range(T):
        for j in range(k):
            if rows[t, j] >= 0:
                assert torch.equal(got[rows[t, j]].view(torch.int16), wide[t, 8:8 + K].cpu().view(torch.int16))
    out = torch.full((T, K + 24), 3.0, device=cuda)
    mb.combine(A, r, out[:, 16:16 + K])
    n = (rows >= 0).sum(1)[:, None]
    assert np.abs(ou.np64(out[:, 16:16 + K]) - n * wv[:, 8:8 + K]).max() <= 3 * 4 * ou.U32 * np.abs(wv).max() * 3
    assert (out[:, :16] == 3).all() and (out[:, 16 + K:] == 3).all()


@pytest.mark.parametrize("T,k,E,K,kind,align", ROW_CASES)
@pytest.mark.parametrize("out_f32", [False, True])
def test_combine_and_gradients(T, k, E, K, kind, align, out_f32, cuda):
    rng = np.random.default_rng(3 * T + K)
    rows, _, src, lead = layout(rng, T, k, E, kind, align)
    R = int(np.prod(lead))
    D, Dv = ou.random_bf16(rng, (R, K))
    D[torch.from_numpy(src) < 0] = float("nan")             # rows of no choice are not read
    w = rng.normal(size=(T, k)).astype(np.float32)
    st = ou.status_word(cuda)
    kind_t = torch.float32 if out_f32 else torch.bfloat16
    r, dD_dev, w_dev = ou.i32(rows, cuda), D.view(lead + (K,)).to(cuda), ou.f32(w, cuda)
    for ww in (w, None):
        out = torch.full((T, K), 7.0, dtype=kind_t, device=cuda)
        mb.combine(dD_dev, r, out, w=None if ww is None else w_dev, status=st)
        ref = oo.combine(Dv, rows, ww)
        mag = oo.combine(np.abs(Dv), rows, None if ww is None else np.abs(ww))
        tol = (k + 1) * ou.U32 * mag + (0 if out_f32 else ou.BF16 * np.abs(ref))
        assert (np.abs(ou.np64(out.float()) - ref) <= tol).all()
    dout = torch.from_numpy(rng.normal(size=(T, K)).astype(np.float32)).to(kind_t)
    dv = ou.np64(dout.float())
    dD = sentinel_like(lead + (K,), cuda)
    keep = dD.clone()
    dw = torch.full((T, k), 9.0, device=cuda)
    mb.combine_backward(dout.to(cuda), dD_dev, r, w_dev, dD, dw, status=st)
    rD, rw = oo.combine_backward(dv, Dv, rows, w)
    got = ou.bf16_np(dD.view(R, K))
    for row in range(R):
        if row in rD:
            assert (np.abs(got[row] - rD[row]) <= (ou.BF16 + 2 * ou.U32) * np.abs(rD[row])).all()
        else:
            assert torch.equal(dD.view(R, K)[row].view(torch.int16), keep.view(R, K)[row].view(torch.int16))
    _, mag = oo.combine_backward(np.abs(dv), np.abs(Dv), rows, w)
    assert (np.abs(ou.np64(dw) - rw) <= K * ou.U32 * mag).all()
    # the rows' gradient alone, with unit weights: dispatch of dout
    dD1 = torch.zeros(lead + (K,), dtype=torch.bfloat16, device=cuda)
    mb.combine_backward(dout.to(cuda), None, r, None, dD1, None, status=st)
    A = torch.zeros(lead + (K,), dtype=torch.bfloat16, device=cuda)
    mb.dispatch(dout.to(torch.bfloat16).to(cuda), r, A, status=st)
    assert torch.equal(dD1.view(torch.int16), A.view(torch.int16))
    assert st.item() == 0


def test_rows_past_the_buffer_are_reported_and_skipped(cuda):
    K = 128
    rows = ou.i32([[0, 4], [5, 3]], cuda)
    x = torch.ones((2, K), dtype=torch.bfloat16, device=cuda)
    buf = torch.zeros((8, K), dtype=torch.bfloat16, device=cuda)
    st = ou.status_word(cuda)
    mb.dispatch(x, rows, buf[:4], status=st)
    assert st.item() == 6 and (buf[4:] == 0).all() and (buf[[0, 3]] == 1).all()
    st.zero_()
    out = torch.zeros((2, K), dtype=torch.bfloat16, device=cuda)
    mb.combine(buf[:4], rows, out, status=st)
    assert st.item() == 6 and (out == 1).all()
    st.zero_()
    dD, dw = torch.zeros((8, K), dtype=torch.bfloat16, device=cuda), torch.zeros((2, 2), device=cuda)
    mb.combine_backward(x, buf[:4], rows, None, dD[:4], dw, status=st)
    assert st.item() == 6 and (dD[4:] == 0).all() and dw.cpu().tolist() == [[128.0, 0.0], [0.0, 128.0]]


def test_offsets_past_2_31_elements(cuda):
    """600000 rows of 4096 columns: rows near the end lie past 2^31 elements."""
    R, K = 600000, 4096
    rng = np.random.default_rng(1)
    x, _ = ou.random_bf16(rng, (2, K))
    x = x.to(cuda)
    rows = ou.i32([[R - 1, 2], [R - 2, -1]], cuda)
    A = torch.empty((R, K), dtype=torch.bfloat16, device=cuda)
    mb.dispatch(x, rows, A)
    assert torch.equal(A[R - 1], x[0]) and torch.equal(A[2], x[0]) and torch.equal(A[R - 2], x[1])
    out = torch.zeros((2, K), dtype=torch.bfloat16, device=cuda)
    mb.combine(A, rows, out)
    assert torch.equal(out[0], 2 * x[0]) and torch.equal(out[1], x[1])
    del A
    Q = torch.empty((R, K), dtype=torch.uint8, device=cuda)
    SF = torch.zeros((1, K // 128, R), dtype=torch.uint8, device=cuda)
    mb.dispatch(x, rows, Q, SFA=SF)
    q, s = oo.quantize(ou.bf16_np(x))
    assert np.array_equal(Q[R - 1].cpu().numpy(), q[0]) and np.array_equal(SF[0, :, R - 1].cpu().numpy(), s[0])
    assert np.array_equal(Q[R - 2].cpu().numpy(), q[1]) and np.array_equal(SF[0, :, R - 2].cpu().numpy(), s[1])


def test_another_stream(cuda):
    rng = np.random.default_rng(8)
    T, k, E, K = 700, 8, 32, 512
    idx = ou.i32(ou.random_choices(rng, T, k, E), cuda)
    x, _ = ou.random_bf16(rng, (T, K))
    x = x.to(cuda)
    cap = T * k + E * 16

    def go(stream):
        rows = torch.empty((T, k), dtype=torch.int32, device=cuda)
        counts = torch.empty(E, dtype=torch.int32, device=cuda)
        work = torch.empty(mb.slots_work_bytes(T * k, E), dtype=torch.uint8, device=cuda)
        A = torch.zeros((cap, K), dtype=torch.uint8, device=cuda)
        SF = torch.zeros((1, K // 128, cap), dtype=torch.uint8, device=cuda)
        out = torch.empty((T, K), dtype=torch.bfloat16, device=cuda)
        back = torch.zeros((cap, K), dtype=torch.bfloat16, device=cuda)
        mb.slots_contiguous(idx, rows, counts, 16, cap, work=work, stream=stream)
        mb.dispatch(x, rows, A, SFA=SF, stream=stream)
        mb.dispatch(x, rows, back, stream=stream)
        mb.combine(back, rows, out, stream=stream)
        return rows, counts, A, SF, out
    first = go(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = go(side)
    side.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_captured_after_copies_and_across_streams(cuda):
    """Slot map and dispatch in a CUDA graph whose nodes before them are a memset
    and a copy, with the tokens written on another stream; replayed with new
    choices and tokens."""
    rng = np.random.default_rng(15)
    T, k, E, K = 600, 8, 16, 256
    cap = T * k + E * 16
    idx_in = torch.empty((T, k), dtype=torch.int32, device=cuda)
    x_in, x = torch.empty((T, K), dtype=torch.bfloat16, device=cuda), torch.empty((T, K), dtype=torch.bfloat16,
                                                                                  device=cuda)
    idx, rows = torch.empty_like(idx_in), torch.empty_like(idx_in)
    counts = torch.empty(E, dtype=torch.int32, device=cuda)
    A, B = torch.empty((cap, K), dtype=torch.bfloat16, device=cuda), torch.empty((cap, K), dtype=torch.bfloat16,
                                                                                 device=cuda)
    work = torch.empty(mb.slots_work_bytes(T * k, E), dtype=torch.uint8, device=cuda)
    st = ou.status_word(cuda)

    def body(main, side):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            x.copy_(x_in)
        st.zero_()
        idx.copy_(idx_in)
        mb.slots_contiguous(idx, rows, counts, 16, cap, work=work, status=st)
        main.wait_stream(side)
        mb.dispatch(x, rows, A, status=st)
        B.copy_(A)
        mb.dispatch(x, rows, B, status=st)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    idx_in.copy_(ou.i32(ou.random_choices(rng, T, k, E), cuda))
    x_in.normal_()
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        body(main, side)
        main.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            body(main, side)
    for _ in range(4):
        choices = ou.random_choices(rng, T, k, E)
        idx_in.copy_(ou.i32(choices, cuda))
        x_in.normal_()
        graph.replay()
        torch.cuda.synchronize()
        want, _, _, _ = oo.slots(choices, E, align_q=16, rows_cap=cap)
        assert st.item() == 0 and np.array_equal(rows.cpu().numpy(), want)
        at = torch.from_numpy(np.argwhere(want >= 0)).to(cuda)
        r = rows[at[:, 0], at[:, 1]].long()
        assert torch.equal(A[r], x_in[at[:, 0]]) and torch.equal(B[r], x_in[at[:, 0]])


@pytest.mark.parametrize("src", ["bf16", "e4m3"])
@pytest.mark.parametrize("kind", ["contiguous", "masked"])
@pytest.mark.parametrize("k,K", [(3, 256), (32, 128), (1, 2176)])
def test_dispatch_of_many_tokens(k, K, kind, src, cuda):
    """Enough tokens that blocks take several each, not a multiple of that; tokens
    without rows, rows at the end of a buffer, and the checkpoint on the way."""
    T, E = 2437, 40
    rng = np.random.default_rng(K + k)
    rows, _, _, lead = layout(rng, T, k, E, kind, 16)
    R, G = int(np.prod(lead)), lead[-1]
    x, xv = ou.random_bf16(rng, (T, K), 3.0)
    q, s = oo.quantize(xv)
    st = ou.status_word(cuda)
    A = torch.full(lead + (K,), 0x7D, dtype=torch.uint8, device=cuda)
    SFA = torch.full((R // G, K // 128, G), 0xEE, dtype=torch.uint8, device=cuda)
    kw = {}
    if src == "bf16":
        X = x.to(cuda)
        kw["CX"] = torch.zeros((T, K), dtype=torch.uint8, device=cuda)
        kw["SCX"] = torch.zeros((T, K // 128), dtype=torch.uint8, device=cuda)
    else:
        X, kw["SX"] = torch.from_numpy(q).to(cuda), torch.from_numpy(s).to(cuda)
    mb.dispatch(X, ou.i32(rows, cuda), A, SFA=SFA, status=st, **kw)
    assert st.item() == 0
    if src == "bf16":
        assert np.array_equal(kw["CX"].cpu().numpy(), q) and np.array_equal(kw["SCX"].cpu().numpy(), s)
    want = np.full((R, K), 0x7D, dtype=np.uint8)
    sf = np.full((R, K // 128), 0xEE, dtype=np.uint8)
    at = np.argwhere(rows >= 0)
    r = rows[at[:, 0], at[:, 1]]
    want[r], sf[r] = q[at[:, 0]], s[at[:, 0]]
    assert np.array_equal(A.view(R, K).cpu().numpy(), want)
    assert np.array_equal(SFA.cpu().numpy().transpose(0, 2, 1).reshape(R, -1), sf)
    bad = ou.i32(np.where(rows == rows.max(), R, rows), cuda)         # one row past the buffer
    A.fill_(0x11)
    mb.dispatch(X, bad, A, SFA=SFA, status=st, **kw)
    assert st.item() == 6
    got = A.view(R, K).cpu().numpy()
    keep = r[r != rows.max()]
    assert np.array_equal(got[keep], want[keep]) and (got[rows.max()] == 0x11).all()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("k,K", [(1, 264), (2, 264), (2, 2176), (3, 1032), (4, 4352), (5, 128), (11, 264)])
def test_combine_of_many_tokens(k, K, f32, cuda):
    """Enough tokens that blocks take several each, not a multiple of that;
    tokens without rows, strided out and dout, a row past the buffer."""
    T, E = 701, 24
    rng = np.random.default_rng(K + k)
    rows, _, src, (R,) = layout(rng, T, k, E, "contiguous", 8)
    D, Dv = ou.random_bf16(rng, (R, K))
    D[torch.from_numpy(src) < 0] = float("nan")
    Dv[src < 0] = 0
    w = rng.normal(size=(T, k)).astype(np.float32)
    kind = torch.float32 if f32 else torch.bfloat16
    st = ou.status_word(cuda)
    r, Dd, wd = ou.i32(rows, cuda), D.to(cuda), ou.f32(w, cuda)
    live = (rows >= 0)[:, :, None]
    V, W = Dv[rows] * live, w.astype(np.float64)[:, :, None]
    out = torch.full((T, K + 8), 7.0, dtype=kind, device=cuda)
    mb.combine(Dd, r, out[:, :K], w=wd, status=st)
    ref, mag = (V * W).sum(1), (np.abs(V) * np.abs(W)).sum(1)
    tol = (k + 1) * ou.U32 * mag + (0 if f32 else ou.BF16 * np.abs(ref))
    assert (np.abs(ou.np64(out[:, :K].float()) - ref) <= tol).all() and (out[:, K:] == 7).all()
    dout = torch.from_numpy(rng.normal(size=(T, K + 16)).astype(np.float32)).to(kind)[:, :K]
    g = ou.np64(dout.float())
    dD, dw = sentinel_like((R, K), cuda), torch.full((T, k), 9.0, device=cuda)
    keep = dD.clone()
    gd = torch.empty((T, K + 16), dtype=kind, device=cuda)[:, :K]
    gd.copy_(dout)
    mb.combine_backward(gd, Dd, r, wd, dD, dw, status=st)
    assert st.item() == 0
    want = np.zeros((R, K))
    want[rows[rows >= 0]] = (g[:, None, :] * W)[rows >= 0]
    got, used = ou.bf16_np(dD), src >= 0
    assert (np.abs(got[used] - want[used]) <= (ou.BF16 + 2 * ou.U32) * np.abs(want[used])).all()
    unused = torch.from_numpy(~used).to(cuda)
    assert torch.equal(dD[unused].view(torch.int16), keep[unused].view(torch.int16))
    dots, mags = (g[:, None, :] * V).sum(2), (np.abs(g[:, None, :]) * np.abs(V)).sum(2)
    assert (np.abs(ou.np64(dw) - dots) <= K * ou.U32 * mags).all()
    t, j = np.argwhere(rows >= 0)[-1]                      # the last choice's row, past the buffer
    bad = rows.copy()
    bad[t, j] = R
    out.fill_(3.0)
    mb.combine(Dd, ou.i32(bad, cuda), out[:, :K], w=wd, status=st)
    assert st.item() == 6
    V[t, j] = 0
    assert (np.abs(ou.np64(out[:, :K].float()) - (V * W).sum(1)) <= tol + ou.BF16 * mag).all()
    st.zero_()
    dw.fill_(9.0)
    mb.combine_backward(gd, Dd, ou.i32(bad, cuda), wd, dD, dw, status=st)
    assert st.item() == 6 and dw[t, j].item() == 0


@pytest.mark.parametrize("T,k,E,M,cap", [
    (0, 2, 3, 4096, None), (1, 1, 1, 70000, None), (7, 3, 5, 4096, None), (7, 2, 200, 1024, None),
    (600, 8, 33, 2048, None), (700, 7, 24, 4096, None),
    (0, 2, 9, None, 40000), (5, 2, 3, None, 100000), (300, 4, 128, None, 50000), (900, 6, 17, None, 70000)])
def test_slots_in_buffers_far_larger_than_the_choices(T, k, E, M, cap, cuda):
    """Most rows hold nothing: every one of them is marked so."""
    idx = ou.random_choices(np.random.default_rng(T + E), T, k, E)
    if M is not None:
        rows, counts, src, st = run_slots(idx, E, cuda, M=M)
        r, c, s, over = oo.slots(idx, E, M_max=M)
    else:
        rows, counts, src, st = run_slots(idx, E, cuda, align=128, cap=cap)
        r, c, s, over = oo.slots(idx, E, align_q=128, rows_cap=cap)
    assert st == 0 and not over
    assert np.array_equal(rows, r) and np.array_equal(counts, c) and np.array_equal(src, s)
