"""Prompts: enough tokens that a warp routes two or four of them at once, not a
multiple of that, and dispatch of wide rows with whole tokens to a block; both
against float64 (the choices and the copies exactly)."""
import numpy as np
import pytest
import torch

from moe_grouped_gemm_side_gb300 import binding as mb
from oracle import ops as oo
from tests import ops_util as ou
from tests.gpu_util import sentinel_like
from tests.test_gpu_k_rows import layout

pytestmark = pytest.mark.gpu

INF = float("inf")
BF, F32 = torch.bfloat16, torch.float32
# Two keys order alike in float64 and on the GPU when they are equal inputs or
# further apart than a score's error and the rounding of its sum with a bias
# (scores up to 1, fewer than 130 units of 2^-24, two keys).
GAP = 2 * 130 * ou.U32


def scores64(x, score):
    if score == "sigmoid":
        return torch.special.expit(x)
    dead = (x == -INF).all(1, keepdim=True)
    return torch.where(dead, torch.zeros_like(x), torch.softmax(torch.where(dead, torch.zeros_like(x), x), 1))


def clear(v, n):
    """Rows whose n largest values, and the one after them, are told apart."""
    v = torch.sort(v, dim=1, descending=True).values[:, :n + 1]
    d = v[:, :-1] - v[:, 1:]
    return ((d == 0) | (d > GAP) | torch.isnan(d)).all(1)


def choose64(x, bias, E, k, score, groups, top_groups, group_top, renorm, scale):
    """idx, w and which rows are clear; NaN counts as -inf."""
    x = torch.where(torch.isnan(x), torch.full_like(x, -INF), x)
    s = scores64(x, score)
    s = torch.where(x == -INF, torch.zeros_like(s), s)
    # without a bias scores compare as logits do: the gaps are those of the logits
    key = torch.where(x == -INF, x, x if bias is None else s + bias)
    fine = torch.ones(x.shape[0], dtype=torch.bool, device=x.device)
    if groups > 1:
        by = torch.where(x == -INF, x, s if bias is None else s + bias).view(-1, groups, E // groups)
        by = torch.sort(by, dim=2, descending=True).values[:, :, :group_top]
        grp = torch.where(torch.isinf(by), torch.zeros_like(by), by).sum(2)
        grp = torch.where(torch.isinf(by[:, :, 0]), torch.full_like(grp, -INF), grp)
        fine &= clear(grp, top_groups)
        rank = torch.argsort(torch.argsort(grp, dim=1, descending=True, stable=True), dim=1)
        key = torch.where((rank >= top_groups).repeat_interleave(E // groups, 1), torch.full_like(key, -INF), key)
    if bias is not None:
        fine &= clear(key, k)
    val, idx = torch.sort(key, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    w = torch.where(val == -INF, torch.zeros_like(val), s.gather(1, idx))
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp(min=2.0 ** -126)
    return torch.where(val == -INF, torch.full_like(idx, -1), idx).int(), w * scale, fine


def prompt(seed, T, E, dtype, pad, device, steps=None):
    """Logits [T, E] in rows E + pad apart: shuffled levels 8 / E apart (or of
    `steps` values, so that experts tie), experts and tokens at -inf."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    order = torch.argsort(torch.rand(T, E, generator=g, device=device), dim=1)
    x = (order % steps).float() / 4 if steps else order * (8.0 / E) - 4
    x[torch.rand(T, E, generator=g, device=device) < 0.02] = -INF
    few = torch.rand(T, generator=g, device=device) < 0.05
    x[few, 3:] = -INF
    x[torch.rand(T, generator=g, device=device) < 0.03] = -INF
    wide = torch.full((T, E + pad), 99.0, dtype=dtype, device=device)
    wide[:, :E] = x.to(dtype)
    return wide


def route(x, bias, c, status):
    T, k = x.shape[0], c["k"]
    idx = torch.full((T, k), -7, dtype=torch.int32, device=x.device)
    w = torch.full((T, k), 9.0, device=x.device)
    mb.route(x, idx, w, score=c["score"], bias=bias, groups=c["groups"], top_groups=c["top_groups"],
             group_top=c["group_top"], renorm=c["renorm"], scale=c["scale"], status=status)
    return idx, w


KEYS = ("E", "k", "score", "groups", "top_groups", "group_top", "renorm", "scale")
CASES = [
    # E, k, score, groups, top_groups, group_top, renorm, scale, bias, dtype, row distance past E
    (64, 8, "softmax", 1, 1, 1, True, 1.0, False, BF, 0),
    (128, 8, "softmax", 1, 1, 1, True, 1.0, False, BF, 8),
    (128, 7, "softmax", 1, 1, 1, True, 2.5, False, BF, 0),
    (256, 8, "sigmoid", 1, 1, 1, True, 1.0, False, BF, 0),
    (200, 5, "sigmoid", 1, 1, 1, False, 1.0, False, BF, 16),
    (96, 3, "softmax", 1, 1, 1, True, 1.0, False, BF, 4),
    (128, 1, "sigmoid", 1, 1, 1, False, 1.0, False, BF, 0),
    (256, 16, "softmax", 1, 1, 1, True, 1.0, False, BF, 0),
    (128, 11, "softmax", 1, 1, 1, True, 1.0, False, BF, 0),
    (256, 17, "softmax", 1, 1, 1, True, 1.0, False, BF, 0),
    (130, 6, "softmax", 1, 1, 1, True, 1.0, False, BF, 1),              # not in whole words
    (160, 6, "softmax", 8, 3, 1, False, 16.0, False, BF, 0),
    (128, 8, "softmax", 1, 1, 1, False, 1.0, False, BF, 0),
    (256, 8, "sigmoid", 8, 4, 2, True, 2.5, True, BF, 0),
    (256, 8, "sigmoid", 8, 4, 2, True, 2.5, True, F32, 0),
    (64, 5, "softmax", 1, 1, 1, True, 1.0, True, F32, 3),
    (60, 4, "softmax", 4, 2, 1, False, 1.0, False, F32, 0),
    (33, 3, "sigmoid", 11, 4, 2, True, 1.0, True, F32, 0),
    (8, 3, "softmax", 1, 1, 1, True, 1.0, False, BF, 0),
    (24, 9, "sigmoid", 1, 1, 1, True, 1.0, True, F32, 1),
    (384, 8, "sigmoid", 8, 4, 2, True, 2.5, True, BF, 0),
    (384, 7, "softmax", 1, 1, 1, True, 1.0, False, F32, 0),
    (300, 4, "softmax", 1, 1, 1, False, 1.0, False, F32, 5),
    (512, 12, "softmax", 1, 1, 1, True, 1.0, False, BF, 0),
    (1000, 3, "sigmoid", 1, 1, 1, False, 1.0, True, F32, 0),
]


def prepare(case, T, device, steps=None):
    E, k, *_, bias, dtype, pad = case
    c = dict(zip(KEYS, case))
    wide = prompt(E + k, T, E, dtype, pad, device, steps)
    b = None
    if bias:
        b = torch.from_numpy(np.round(np.random.default_rng(E).normal(size=E) * 20) / 1024).to(device)
    idx, w, fine = choose64(wide[:, :E].double(), b, **c)
    # rows that hang on a rounding give way to others
    at, bad = fine.nonzero().flatten(), (~fine).nonzero().flatten()
    assert at.numel() > T // 2
    swap = at[torch.arange(bad.numel(), device=device) % at.numel()]
    for t in (wide, idx, w):
        t[bad] = t[swap]
    return c, wide, None if b is None else b.float(), idx, w


@pytest.mark.parametrize("T", [10007, 20011])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"E{c[0]}k{c[1]}{c[2]}g{c[3]}{'b' if c[8] else ''}{c[9]}"[:-4])
def test_prompt(case, T, cuda):
    c, wide, bias, ridx, rw = prepare(case, T, cuda)
    E, st = c["E"], ou.status_word(cuda)
    idx, w = route(wide[:, :E], bias, c, st)
    assert st.item() == 0 and torch.equal(idx, ridx)
    assert ((w.double() - rw).abs() <= 3 * ou.score_tol(16.0, E) * rw).all()
    # the same bits for a token wherever it stands among others
    idx2, w2 = route(wide[1:, :E].contiguous(), bias, c, st)
    assert torch.equal(idx2, ridx[1:]) and torch.equal(w2, w[1:])
    # NaN in one expert of some tokens: reported, never chosen, the others as before
    hit = torch.arange(5, T, 7, device=cuda)
    at = (hit * 31) % E
    wide[hit, at] = float("nan")
    nidx, nw, fine = choose64(wide[:, :E].double(), None if bias is None else bias.double(), **c)
    idx3, w3 = route(wide[:, :E], bias, c, st)
    assert st.item() == 6
    same = torch.ones(T, dtype=torch.bool, device=cuda)
    same[hit] = False
    assert torch.equal(idx3[same], idx[same]) and torch.equal(w3[same], w[same])
    assert torch.equal(idx3[fine], nidx[fine]) and torch.isfinite(w3).all()


@pytest.mark.parametrize("E,k,dtype,pad", [(128, 8, BF, 0), (256, 7, BF, 0), (64, 5, BF, 0), (384, 6, BF, 0),
                                           (96, 8, F32, 0), (256, 8, F32, 1)])
def test_ties_go_to_the_lowest_expert(E, k, dtype, pad, cuda):
    case = (E, k, "softmax", 1, 1, 1, True, 1.0, False, dtype, pad)
    c, wide, _, ridx, rw = prepare(case, 20011, cuda, steps=6)
    idx, w = route(wide[:, :E], None, c, None)
    assert torch.equal(idx, ridx)
    assert ((w.double() - rw).abs() <= 3 * ou.score_tol(16.0, E) * rw).all()


@pytest.mark.parametrize("src,dst", [("bf16", "bf16"), ("bf16", "e4m3"), ("e4m3", "bf16"), ("e4m3", "e4m3")])
@pytest.mark.parametrize("k,K", [(3, 5120), (2, 7168), (1, 8192), (2, 9216)])
def test_dispatch_of_many_wide_tokens(k, K, src, dst, cuda):
    """Whole tokens to a block, three and four passes of its threads, and a token
    in two blocks; the checkpoint on the way."""
    T, E = 613, 24
    rng = np.random.default_rng(K + k)
    rows, _, _, (R,) = layout(rng, T, k, E, "contiguous", 16)
    x, xv = ou.random_bf16(rng, (T, K), 3.0)
    q, s = oo.quantize(xv)
    st = ou.status_word(cuda)
    kw = {}
    if dst == "e4m3":
        A, kw["SFA"] = torch.full((R, K), 0x7D, dtype=torch.uint8, device=cuda), \
            torch.full((K // 128, R), 0xEE, dtype=torch.uint8, device=cuda)
        want, sf = torch.full((R, K), 0x7D, dtype=torch.uint8), np.full((R, K // 128), 0xEE, dtype=np.uint8)
    else:
        A = sentinel_like((R, K), cuda)
        want, sf = A.cpu(), None
    if src == "bf16":
        X = x.to(cuda)
        kw["CX"] = torch.zeros((T, K), dtype=torch.uint8, device=cuda)
        kw["SCX"] = torch.zeros((T, K // 128), dtype=torch.uint8, device=cuda)
    else:
        X, kw["SX"] = torch.from_numpy(q).to(cuda), torch.from_numpy(s).to(cuda)
    mb.dispatch(X, ou.i32(rows, cuda), A, status=st, **kw)
    assert st.item() == 0
    at = np.argwhere(rows >= 0)
    r, t = torch.from_numpy(rows[at[:, 0], at[:, 1]]), torch.from_numpy(at[:, 0])
    if dst == "e4m3":
        want[r], sf[r.numpy()] = torch.from_numpy(q)[t], s[at[:, 0]]
        assert np.array_equal(kw["SFA"].cpu().numpy().T, sf)
    else:
        want[r] = (x if src == "bf16" else torch.from_numpy(oo.dequantize(q, s)).to(BF))[t]
    assert torch.equal(A.cpu().view(torch.uint8), want.view(torch.uint8))
    if src == "bf16":
        assert np.array_equal(kw["CX"].cpu().numpy(), q) and np.array_equal(kw["SCX"].cpu().numpy(), s)
