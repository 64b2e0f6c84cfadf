"""Routing and its gradient on the GPU against the float64 oracle: choices
exactly, weights and gradients to the bounds of tests/ops_util.py."""
import itertools

import numpy as np
import pytest
import torch

from moe_grouped_gemm_side_gb300 import binding as mb
from oracle import ops as oo
from tests import ops_util as ou

pytestmark = pytest.mark.gpu


def make_logits(seed, T, E, dtype, c, bias):
    """Rows whose experts differ by well more than a rounding (or tie exactly),
    so that the choice does not hang on the last bit of a score."""
    rows, x = [], None
    for t in range(T):
        for s in itertools.count():
            rng = np.random.default_rng([seed, t, s])
            x = (rng.permutation(E) * (8.0 / E) - 4.0 + rng.normal() * 0.5).astype(np.float32)
            if rng.random() < 0.3:
                x[rng.random(E) < 0.2] = -np.inf
            v = torch.from_numpy(x).to(dtype)
            _, _, gap = oo.route(v.float().numpy()[None], c["k"], c["score"], bias, c["groups"], c["top_groups"],
                                 c["group_top"])
            if gap[0] > 1e-6:
                break
        rows.append(v)
    return torch.stack(rows)


CASES = [
    # T, E, k, score, groups, top_groups, group_top, bias, renorm, scale, dtype
    (1, 1, 1, "softmax", 1, 1, 1, False, True, 1.0, torch.float32),
    (3, 2, 2, "sigmoid", 1, 1, 1, True, False, 1.0, torch.bfloat16),
    (7, 3, 2, "softmax", 3, 2, 1, False, False, 2.0, torch.float32),
    (9, 8, 2, "softmax", 1, 1, 1, False, True, 1.0, torch.bfloat16),
    (5, 31, 4, "sigmoid", 1, 1, 1, True, True, 2.5, torch.float32),
    (5, 33, 5, "softmax", 11, 4, 2, True, True, 1.0, torch.float32),
    (4, 60, 4, "softmax", 4, 2, 1, False, False, 1.0, torch.bfloat16),
    (40, 64, 6, "softmax", 1, 1, 1, False, False, 16.0, torch.bfloat16),
    (17, 100, 7, "sigmoid", 5, 3, 2, True, True, 1.0, torch.float32),
    (33, 128, 8, "softmax", 1, 1, 1, True, True, 1.0, torch.bfloat16),
    (12, 160, 6, "softmax", 8, 3, 1, False, False, 16.0, torch.float32),
    (19, 256, 8, "sigmoid", 8, 4, 2, True, True, 2.5, torch.float32),
    (6, 256, 8, "sigmoid", 32, 4, 2, False, True, 1.0, torch.bfloat16),
    (5, 257, 3, "softmax", 1, 1, 1, False, True, 1.0, torch.float32),
    (4, 384, 12, "sigmoid", 2, 1, 2, False, False, 1.0, torch.float32),
    (5, 384, 8, "sigmoid", 8, 4, 2, True, True, 2.5, torch.bfloat16),
    (4, 300, 5, "softmax", 1, 1, 1, False, False, 1.0, torch.bfloat16),
    (4, 500, 8, "softmax", 1, 1, 1, True, True, 1.0, torch.bfloat16),
    (3, 1000, 32, "softmax", 1, 1, 1, False, True, 1.0, torch.float32),
    (2, 1024, 32, "sigmoid", 16, 5, 2, False, True, 1.0, torch.float32),
    (2, 20, 20, "softmax", 1, 1, 1, False, True, 1.0, torch.float32),
]


def case_dict(c):
    return dict(zip(("T", "E", "k", "score", "groups", "top_groups", "group_top", "bias", "renorm", "scale", "dtype"),
                    c))


def run_route(c, logits, bias, device, status=None, stream=None):
    T, k = logits.shape[0], c["k"]
    idx = torch.full((T, k), -7, dtype=torch.int32, device=device)
    w = torch.full((T, k), 9.0, device=device)
    mb.route(logits, idx, w, score=c["score"], bias=bias, groups=c["groups"], top_groups=c["top_groups"],
             group_top=c["group_top"], renorm=c["renorm"], scale=c["scale"], status=status, stream=stream)
    return idx, w


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"E{c[1]}k{c[2]}{c[3]}g{c[4]}")
def test_route_and_gradient(case, cuda):
    c = case_dict(case)
    T, E, k = c["T"], c["E"], c["k"]
    rng = np.random.default_rng(17 * E + k)
    bias = np.round(rng.normal(size=E) * 20) / 1024 if c["bias"] else None
    logits = make_logits(E, T, E, c["dtype"], c, bias)
    x = logits.float().numpy().astype(np.float64)
    st = ou.status_word(cuda)
    dev = logits.to(cuda)
    idx, w = run_route(c, dev, None if bias is None else ou.f32(bias, cuda), cuda, st)
    ridx, rw, gap = oo.route(x, k, c["score"], bias, c["groups"], c["top_groups"], c["group_top"], c["renorm"],
                             c["scale"])
    assert gap.min() > 1e-6
    assert st.item() == 0
    assert np.array_equal(idx.cpu().numpy(), ridx)
    tol = ou.score_tol(16.0, E)
    assert (np.abs(ou.np64(w) - rw) <= 3 * tol * np.abs(rw)).all()

    dw = rng.normal(size=(T, k)).astype(np.float32)
    dl = torch.full_like(dev, 5.0)
    mb.route_backward(dev, idx, ou.f32(dw, cuda), dl, score=c["score"], renorm=c["renorm"], scale=c["scale"],
                      status=st)
    ref = oo.route_backward(x, ridx, dw, c["score"], c["renorm"], c["scale"])
    got = ou.np64(dl.float())
    # every term of the gradient is at most scale * max|dw| * s_e in size
    big = np.stack([oo.scores(r, c["score"])[0] for r in x])
    if c["renorm"]:
        big = big / np.maximum([[big[t][ridx[t][ridx[t] >= 0]].sum()] for t in range(T)], 1e-30)
    bound = 8 * tol * c["scale"] * np.abs(dw).max() * big * k + 1e-30
    if c["dtype"] == torch.bfloat16:
        bound = bound + ou.BF16 * np.abs(ref)
    assert st.item() == 0
    assert (np.abs(got - ref) <= bound).all()
    assert np.isfinite(got).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_with_nothing_left(score, dtype, cuda):
    """-inf everywhere, fewer live experts than choices, the type's lowest
    value, +inf, and equal logits; finite results throughout."""
    inf, low = float("inf"), torch.finfo(dtype).min
    E, k = 40, 4
    x = torch.zeros(7, E)
    x[0] = -inf
    x[1] = -inf
    x[1, 33] = 1.0
    x[2] = -inf
    x[2, [5, 39]] = torch.tensor([-3.0, 2.0])
    x[3] = low
    x[4] = low
    x[4, 17] = 0.0
    x[5, [9, 30]] = inf
    x = x.to(dtype).to(cuda)
    st = ou.status_word(cuda)
    c = dict(k=k, score=score, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0)
    idx, w = run_route(c, x, None, cuda, st)
    idx, w = idx.cpu(), w.cpu()
    assert st.item() == 0
    assert idx[0].tolist() == [-1] * 4 and w[0].tolist() == [0.0] * 4
    assert idx[1].tolist() == [33, -1, -1, -1] and w[1].tolist() == [1.0, 0.0, 0.0, 0.0]
    assert idx[2].tolist() == [39, 5, -1, -1]
    assert idx[3].tolist() == [0, 1, 2, 3]
    assert idx[4].tolist() == [17, 0, 1, 2] and w[4, 0] == 1.0
    assert idx[5].tolist() == [9, 30, 0, 1]
    assert idx[6].tolist() == [0, 1, 2, 3] and torch.allclose(w[6], torch.full((4,), 0.25))
    assert torch.isfinite(w).all()
    for renorm in (True, False):
        dl = torch.full_like(x, 3.0)
        mb.route_backward(x, idx.to(cuda), torch.ones(7, k, device=cuda), dl, score=score, renorm=renorm, status=st)
        assert torch.isfinite(dl.float()).all()
        assert (dl[0] == 0).all()
        assert (dl[1, :33] == 0).all() and (dl[1, 34:] == 0).all()
    assert st.item() == 0


@pytest.mark.parametrize("width", [128, 137])
def test_infinity_beside_the_largest_bf16_and_zeros_of_both_signs(width, cuda):
    """+inf counts as the largest fp32 value, so it beats bf16's largest; -0 and 0
    are one value, whole rows (width 128) or not."""
    big = torch.finfo(torch.bfloat16).max
    x = torch.full((2, width), -5.0, dtype=torch.bfloat16, device=cuda)
    x = x[:, :128]
    x[0, 7], x[0, 3], x[0, 100] = float("inf"), big, float("inf")
    x[1, 9], x[1, 4], x[1, 70] = 0.0, -0.0, -0.0
    c = dict(k=3, score="softmax", groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0)
    idx, w = run_route(c, x, None, cuda)
    assert idx.cpu().tolist() == [[7, 100, 3], [4, 9, 70]]
    assert w[0].cpu().tolist() == [0.5, 0.5, 0.0] and torch.allclose(w[1], torch.full((3,), 1 / 3, device=cuda))


def test_nan_is_reported_and_never_chosen(cuda):
    x = torch.zeros(3, 50, device=cuda)
    x[1, 0] = float("nan")
    st = ou.status_word(cuda)
    c = dict(k=2, score="sigmoid", groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0)
    for y in (x, x.to(torch.bfloat16), torch.cat([x, x], 1).to(torch.bfloat16)[:, :50]):
        st.zero_()
        idx, w = run_route(c, y, None, cuda, st)
        assert st.item() == 6 and idx.cpu().tolist() == [[0, 1], [1, 2], [0, 1]] and torch.isfinite(w).all()


def test_bias_of_minus_infinity_closes_an_expert(cuda):
    x = torch.zeros(2, 64, device=cuda)
    b = torch.zeros(64, device=cuda)
    b[[0, 2]] = float("-inf")
    c = dict(k=3, score="softmax", groups=1, top_groups=1, group_top=1, renorm=False, scale=1.0)
    idx, _ = run_route(c, x, b, cuda)
    assert idx.cpu().tolist() == [[1, 3, 4]] * 2


def test_strided_rows_streams_and_repeats(cuda):
    """Rows further apart than E (odd distance: no vector alignment), another
    stream, no tokens, and the same bits on every run."""
    T, E = 300, 61
    rng = np.random.default_rng(4)
    wide = torch.from_numpy(rng.normal(size=(T, 77)).astype(np.float32)).to(torch.bfloat16).to(cuda)
    view = wide[:, 5:5 + E]
    c = dict(k=3, score="softmax", groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0)
    idx, w = run_route(c, view, None, cuda)
    idx2, w2 = run_route(c, view.contiguous(), None, cuda)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        idx3, w3 = run_route(c, view, None, cuda, stream=side)
    side.synchronize()
    assert torch.equal(idx, idx2) and torch.equal(w, w2) and torch.equal(idx, idx3) and torch.equal(w, w3)
    out = torch.full((T, 90), 7.0, dtype=torch.bfloat16, device=cuda)
    dw = torch.from_numpy(rng.normal(size=(T, 3)).astype(np.float32)).to(cuda)
    mb.route_backward(view, idx, dw, out[:, 8:8 + E], renorm=True)
    ref = torch.empty((T, E), dtype=torch.bfloat16, device=cuda)
    mb.route_backward(view.contiguous(), idx, dw, ref, renorm=True)
    assert torch.equal(out[:, 8:8 + E], ref)
    assert (out[:, :8] == 7).all() and (out[:, 8 + E:] == 7).all()
    idx0, w0 = run_route(c, view[:0], None, cuda)
    assert idx0.shape == (0, 3)


def test_backward_refuses_bad_choices_on_the_device(cuda):
    x = torch.zeros(2, 8, device=cuda)
    idx = torch.tensor([[1, 8], [-2, 3]], dtype=torch.int32, device=cuda)
    st = ou.status_word(cuda)
    dl = torch.empty_like(x)
    mb.route_backward(x, idx, torch.ones(2, 2, device=cuda), dl, score="sigmoid", status=st)
    assert st.item() == 6
    assert (dl.cpu() != 0).nonzero().tolist() == [[0, 1], [1, 3]]


def test_gradient_against_differences(cuda):
    """Central differences of the kernel's own weights in fp32: step 2^-5 leaves
    a truncation error of h^2 / 6 |w'''| <= 2^-10 / 6 * scale-free third
    derivatives below 1, and a rounding error of about 2^-23 / h."""
    T, E, k = 4, 24, 3
    rng = np.random.default_rng(9)
    x = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32) * 2).to(cuda)
    for score in ("softmax", "sigmoid"):
        c = dict(k=k, score=score, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0)
        idx, _ = run_route(c, x, None, cuda)
        dw = torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32)).to(cuda)
        dl = torch.empty_like(x)
        mb.route_backward(x, idx, dw, dl, score=score, renorm=True)
        h = 2.0 ** -5
        for j in range(k):
            e = idx[:, j].long()
            probe = []
            for sign in (1, -1):
                y = x.scatter_add(1, e[:, None], torch.full((T, 1), sign * h, device=cuda))
                # the choices stay: everything else is masked
                keep = torch.full_like(y, float("-inf")).scatter(1, idx.long(), y.gather(1, idx.long()))
                i2, w2 = run_route(c, keep, None, cuda)
                at = (i2[:, :, None] == idx[:, None, :]).float()
                probe.append((w2[:, :, None] * at * dw[:, None, :]).sum((1, 2)))
            diff = (probe[0] - probe[1]) / (2 * h)
            got = dl.gather(1, e[:, None])[:, 0]
            assert (diff - got).abs().max() < 2.0 ** -10 / 6 * 4 * dw.abs().sum(1).max() + 2.0 ** -16


@pytest.mark.parametrize("case", [
    (6, 66, 5, "softmax", 22, 9, 2, True, True, 1.0, torch.float32),         # groups smaller than a lane's experts
    (6, 100, 4, "sigmoid", 20, 7, 1, False, True, 1.0, torch.bfloat16),
    (9, 30, 3, "softmax", 3, 2, 1, False, True, 1.0, torch.bfloat16),        # one expert a lane
    (9, 192, 8, "sigmoid", 4, 2, 2, True, True, 1.0, torch.bfloat16),
    (5, 336, 6, "softmax", 12, 5, 1, False, False, 1.0, torch.float32),
    (4, 1000, 9, "sigmoid", 8, 3, 2, True, False, 2.0, torch.float32),
], ids=lambda c: f"E{c[1]}g{c[4]}")
def test_groups_of_any_size(case, cuda):
    test_route_and_gradient(case, cuda)


@pytest.mark.parametrize("E,k,score,renorm,dtype", [
    (40, 8, "softmax", True, torch.bfloat16), (100, 7, "sigmoid", True, torch.float32),
    (129, 3, "sigmoid", False, torch.bfloat16), (9, 2, "softmax", True, torch.float32),
    (300, 4, "sigmoid", True, torch.bfloat16), (24, 9, "softmax", True, torch.float32)])
def test_gradient_of_many_tokens(E, k, score, renorm, dtype, cuda):
    """Enough tokens that a warp takes several, not a multiple of that: any
    valid choices, with experts chosen twice, choices left out and tokens
    without one; strided rows; a choice past the experts reported and skipped."""
    T = 20011
    rng = np.random.default_rng(E)
    x = torch.from_numpy(rng.normal(size=(T, E + 8)).astype(np.float32)).to(dtype)
    idx = rng.integers(0, E, size=(T, k))
    idx[rng.random((T, k)) < 0.1] = -1
    idx[rng.random(T) < 0.05] = -1
    dw = rng.normal(size=(T, k)).astype(np.float32)
    dev = x.to(cuda)
    dl = torch.full((T, E + 16), 5.0, dtype=dtype, device=cuda)
    st = ou.status_word(cuda)
    mb.route_backward(dev[:, :E], ou.i32(idx, cuda), ou.f32(dw, cuda), dl[:, :E], score=score, renorm=renorm,
                      scale=2.0, status=st)
    assert st.item() == 0 and (dl[:, E:] == 5).all()
    v = x.float().numpy()[:, :E].astype(np.float64)
    ref = oo.route_backward(v, idx, dw, score, renorm, 2.0)
    got = ou.np64(dl[:, :E].float())
    chosen = np.zeros((T, E + 1), dtype=bool)
    np.put_along_axis(chosen, np.where(idx < 0, E, idx), True, 1)
    assert (got[~chosen[:, :E]] == 0).all()
    # k terms, each at most scale * max|dw|, off by the errors of three scores
    bound = 8 * ou.score_tol(16.0, E) * 2.0 * np.abs(dw).max() * k
    assert (np.abs(got - ref) <= bound + (ou.BF16 * np.abs(ref) if dtype == torch.bfloat16 else 0)).all()
    bad = idx.copy()
    bad[T - 1], bad[T - 2, 0] = -1, E
    mb.route_backward(dev[:, :E], ou.i32(bad, cuda), ou.f32(dw, cuda), dl[:, :E], score=score, renorm=renorm,
                      scale=2.0, status=st)
    assert st.item() == 6 and (dl[T - 1, :E] == 0).all()
    assert torch.equal(dl[:T - 2, :E], torch.from_numpy(got[:T - 2]).to(dtype).to(cuda))
