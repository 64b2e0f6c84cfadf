"""Pins of oracle/ops.py: hand-worked routings and slot maps, the slot map
against the planning oracle, quantisation against its definition, and every
gradient against central differences of the forward functions."""
import numpy as np
import pytest

from oracle import numerics as on
from oracle import ops as oo
from oracle import plan as op

pytestmark = pytest.mark.cpu


def test_route_by_hand():
    x = np.log(np.array([[1.0, 4.0, 2.0, 1.0]]))
    idx, w, _ = oo.route(x, 2, "softmax")
    assert idx.tolist() == [[1, 2]] and np.allclose(w, [[0.5, 0.25]])
    idx, w, _ = oo.route(x, 2, "softmax", renorm=True, scale=3.0)
    assert np.allclose(w, [[2.0, 1.0]])
    # ties: the lowest expert; the bias changes the choice and not the weight
    idx, w, _ = oo.route(x, 4, "softmax")
    assert idx.tolist() == [[1, 2, 0, 3]]
    idx, w, _ = oo.route(x, 1, "softmax", bias=[0, 0, 0, 1.0])
    assert idx.tolist() == [[3]] and np.allclose(w, [[0.125]])
    assert np.allclose(oo.route(np.zeros((1, 2)), 1, "sigmoid")[1], [[0.5]])


def test_route_masked_rows_and_groups():
    inf = np.inf
    idx, w, _ = oo.route([[-inf, -inf, 0.0, -inf]], 2, "softmax", renorm=True)
    assert idx.tolist() == [[2, -1]] and w.tolist() == [[1.0, 0.0]]
    idx, w, _ = oo.route([[-inf] * 4], 2, "softmax", renorm=True)
    assert idx.tolist() == [[-1, -1]] and w.tolist() == [[0.0, 0.0]]
    idx, _, _ = oo.route([[np.nan, 1.0, 0.0, -1.0]], 4, "sigmoid")
    assert idx.tolist() == [[1, 2, 3, -1]]
    # groups of two; sums of two: 0.5+0.5 < 0.9+0.3, but the single best is in group 1 either way
    x = np.array([[0.5, 0.5, 0.9, 0.3, 0.8, -inf]])
    key = np.array([[np.log(v / (1 - v)) if v > 0 else -inf for v in x[0]]])     # sigmoid gives x back
    idx, _, _ = oo.route(key, 2, "sigmoid", groups=3, top_groups=1, group_top=2)
    assert idx.tolist() == [[2, 3]]
    idx, _, _ = oo.route(key, 3, "sigmoid", groups=3, top_groups=2, group_top=1)
    assert idx.tolist() == [[2, 4, 3]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_is_the_derivative(score, renorm):
    rng = np.random.default_rng(7)
    x = rng.normal(size=(5, 9))
    x[1, 3] = -np.inf
    idx, _, _ = oo.route(x, 4, score)
    idx[2, 3] = -1
    dw = rng.normal(size=idx.shape)
    dx = oo.route_backward(x, idx, dw, score, renorm, 1.7)
    h = 1e-6
    for t in range(5):
        for e in range(9):
            if not np.isfinite(x[t, e]):
                assert dx[t, e] == 0
                continue
            a, b = x.copy(), x.copy()
            a[t, e] += h
            b[t, e] -= h
            diff = ((oo.route_weights(a, idx, score, renorm, 1.7) - oo.route_weights(b, idx, score, renorm, 1.7))
                    * dw).sum() / (2 * h)
            assert abs(diff - dx[t, e]) < 1e-8


def test_slots_by_hand_and_against_the_plan():
    idx = np.array([[0, 2], [2, -1], [0, 2]])
    rows, counts, src, over = oo.slots(idx, 3, align_q=4, rows_cap=8)
    assert rows.tolist() == [[0, 4], [5, -1], [1, 6]] and counts.tolist() == [2, 0, 3] and not over
    assert src.tolist() == [0, 4, -1, -1, 1, 2, 5, -1]
    rows, counts, src, over = oo.slots(idx, 3, align_q=4, rows_cap=6)        # expert 2 does not fit
    assert rows.tolist() == [[0, -1], [-1, -1], [1, -1]] and over and src.tolist() == [0, 4] + [-1] * 4
    rows, counts, src, over = oo.slots(idx, 3, M_max=2)
    assert rows.tolist() == [[0, 4], [5, -1], [1, -1]] and counts.tolist() == [2, 0, 2] and over
    rng = np.random.default_rng(3)
    for q in (1, 8, 16):
        idx = rng.integers(-1, 11, size=(57, 3))
        cap = 57 * 3 + 11 * q
        rows, counts, src, over = oo.slots(idx, 11, align_q=q, rows_cap=cap)
        p = op.plan(counts.tolist(), q)
        assert not over
        for e in range(11):
            got = src[p.offsets[e]:p.offsets[e] + counts[e]]
            assert (idx.reshape(-1)[got] == e).all() and (np.diff(got) > 0).all()
        assert (src[p.P:] == -1).all() and (src >= 0).sum() == (idx >= 0).sum()


def test_quantize_is_the_nearest_code_of_the_smallest_scale():
    rng = np.random.default_rng(5)
    x = rng.normal(size=(6, 256)) * np.exp2(rng.integers(-30, 30, size=(6, 1)))
    x[0, :128] = 0
    x[1, 5] = 448.0 * 2.0 ** 20
    x[2, 7] = np.nextafter(448.0 * 2.0 ** 31, np.inf)      # a hair above: the next scale
    codes, sf = oo.quantize(x)
    y = oo.dequantize(codes, sf)
    assert sf[0, 0] == 127 and sf[1, 0] == 147 and sf[2, 0] == 159
    grid = np.concatenate([-oo.E4M3_GRID[::-1], oo.E4M3_GRID])
    for r in range(6):
        for b in range(2):
            s = 2.0 ** (int(sf[r, b]) - 127)
            v = x[r, 128 * b:128 * b + 128]
            best = np.abs(v[:, None] - s * grid[None]).min(1)
            assert np.array_equal(np.abs(y[r, 128 * b:128 * b + 128] - v), best)
            if np.abs(v).max() > 0:
                assert 448 * s / 2 < np.abs(v).max() <= 448 * s
    assert np.array_equal(on.decode_e4m3(np.arange(127, dtype=np.uint8)), oo.E4M3_GRID)


def test_swiglu_backward_is_the_derivative():
    rng = np.random.default_rng(11)
    h = rng.normal(size=(3, 256)) * 2
    dy, w = rng.normal(size=(3, 128)), rng.normal(size=3)
    dh, y, dw = oo.swiglu_backward(dy, h, w)
    assert np.allclose(y, oo.swiglu(h) * w[:, None]) and np.allclose(dw, (dy * oo.swiglu(h)).sum(1))
    eps = 1e-6
    for r, c in [(0, 0), (0, 130), (1, 127), (2, 128), (2, 255)]:
        a, b = h.copy(), h.copy()
        a[r, c] += eps
        b[r, c] -= eps
        diff = ((oo.swiglu(a) - oo.swiglu(b)) * dy * w[:, None]).sum() / (2 * eps)
        assert abs(diff - dh[r, c]) < 1e-8


def test_combine_and_its_gradients():
    rng = np.random.default_rng(13)
    D, rows, w = rng.normal(size=(7, 8)), np.array([[0, 3], [-1, 5], [-1, -1]]), rng.normal(size=(3, 2))
    out = oo.combine(D, rows, w)
    assert np.allclose(out[0], w[0, 0] * D[0] + w[0, 1] * D[3]) and np.allclose(out[1], w[1, 1] * D[5])
    assert (out[2] == 0).all()
    dout = rng.normal(size=(3, 8))
    dD, dw = oo.combine_backward(dout, D, rows, w)
    assert sorted(dD) == [0, 3, 5] and (dw[2] == 0).all() and dw[1, 0] == 0
    eps = 1e-6
    for r in (0, 5):
        for c in (0, 7):
            a = D.copy()
            a[r, c] += eps
            assert abs(((oo.combine(a, rows, w) - out) * dout).sum() / eps - dD[r][c]) < 1e-8
    a = w.copy()
    a[1, 1] += eps
    assert abs(((oo.combine(D, rows, a) - out) * dout).sum() / eps - dw[1, 1]) < 1e-8
