"""The operators around the grouped GEMMs in float64: routing and its
gradient, the slot map, dispatch, combine and its gradients, and SwiGLU with
its 8-bit checkpoint and backward pass.  Plain loops over tokens and rows,
written from the definitions; codes and scales go through the oracle's own
E4M3 / UE8M0 decoding."""
import math

import numpy as np

from . import numerics as on

E4M3_MAX = 448.0
# every non-negative finite E4M3 value in code order: codes 0..126
E4M3_GRID = on.decode_e4m3(np.arange(127, dtype=np.uint8)).astype(np.float64)


# ------------------------------------------------------------------ routing
def scores(x, score):
    """float64 scores of logits x [E]; an expert at -inf (or NaN) scores 0."""
    x = np.asarray(x, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    live = x != -np.inf
    s = np.zeros_like(x)
    if score == "sigmoid":
        s[live] = [1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 for v in x[live]]
    elif live.any():
        e = np.exp(x[live] - x[live].max())
        s[live] = e / e.sum()
    return s, live


def route(x, k, score, bias=None, groups=1, top_groups=1, group_top=1, renorm=False, scale=1.0):
    """(idx [T, k], w [T, k], gap [T]): gap is the smallest non-zero distance
    that any comparison next to a cut saw (inf if there was none)."""
    x = np.asarray(x, dtype=np.float64)
    T, E = x.shape
    idx = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    gap = np.full(T, np.inf)

    def cut(pairs, n, t):
        """The n largest (value, index) pairs: value descending, index ascending."""
        pairs = sorted(pairs, key=lambda p: (-p[0], p[1]))
        for a, b in zip(pairs[:n + 1], pairs[1:n + 1]):
            if a[0] != b[0]:
                gap[t] = min(gap[t], a[0] - b[0])
        return pairs[:n]
    for t in range(T):
        s, live = scores(x[t], score)
        key = s + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
        live = live & (key != -np.inf) & ~np.isnan(key)
        ok = set(np.nonzero(live)[0].tolist())
        if groups > 1:
            gs = E // groups
            gsc = []
            for g in range(groups):
                mem = sorted((key[e] for e in range(g * gs, (g + 1) * gs) if e in ok), reverse=True)
                gsc.append((sum(mem[:group_top]) if mem else -np.inf, g))
            stay = {g for _, g in cut(gsc, top_groups, t)}
            ok = {e for e in ok if e // gs in stay}
        for j, (_, e) in enumerate(cut([(key[e], e) for e in ok], k, t)):
            idx[t, j], w[t, j] = e, s[e]
        if renorm and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return idx, w * scale, gap


def route_weights(x, idx, score, renorm, scale):
    """Weights [T, k] of given choices (what the gradient differentiates)."""
    w = np.zeros(idx.shape)
    for t in range(idx.shape[0]):
        s, _ = scores(x[t], score)
        w[t] = [s[e] if e >= 0 else 0.0 for e in idx[t]]
        if renorm and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return w * scale


def route_backward(x, idx, dw, score, renorm, scale):
    x, dw = np.asarray(x, dtype=np.float64), np.asarray(dw, dtype=np.float64)
    T, E = x.shape
    dx = np.zeros((T, E))
    for t in range(T):
        s, _ = scores(x[t], score)
        at = [j for j in range(idx.shape[1]) if idx[t, j] >= 0]
        e = idx[t, at].astype(int)
        ds = scale * dw[t, at]                      # by the (renormalised) score
        total = s[e].sum()
        if renorm:
            ds = (ds - (ds * s[e]).sum() / total) / total if total > 0 else np.zeros(len(at))
        full = np.zeros(E)
        for i, d in zip(e, ds):
            full[i] += d
        dx[t] = full * s * (1.0 - s) if score == "sigmoid" else s * (full - (full * s).sum())
    return dx


# ------------------------------------------------------------------ slot map
def slots(idx, E, align_q=None, rows_cap=None, M_max=None):
    """(rows [T, k], counts [E], src [rows], overflow) of the contiguous layout
    (align_q, rows_cap) or the masked one (M_max)."""
    flat = [int(e) if 0 <= e < E else -1 for e in np.asarray(idx).reshape(-1)]
    of = [[i for i, f in enumerate(flat) if f == e] for e in range(E)]
    total = E * M_max if M_max is not None else rows_cap
    rows, src, counts, overflow = [-1] * len(flat), [-1] * total, [], False
    start = 0
    for e in range(E):
        n = len(of[e])
        if M_max is not None:
            base, take = e * M_max, min(n, M_max)
            overflow |= n > M_max
            counts.append(take)
        else:
            base, take = start, n if start + n <= rows_cap else 0
            start += -(-n // align_q) * align_q
            overflow |= start > rows_cap
            counts.append(n)
        for i in range(take):
            rows[of[e][i]] = base + i
            src[base + i] = of[e][i]
    return (np.array(rows, dtype=np.int64).reshape(np.shape(idx)), np.array(counts), np.array(src), overflow)


# --------------------------------------------------------------- checkpoints
def quantize(x):
    """(codes uint8 [R, C], scales uint8 [R, C/128]) of float64 x, by search: the
    smallest scale that holds the block, the nearest code, ties to even."""
    R, C = x.shape
    codes = np.zeros((R, C), dtype=np.uint8)
    sf = np.zeros((R, C // 128), dtype=np.uint8)
    for r in range(R):
        for b in range(C // 128):
            v = x[r, 128 * b:128 * b + 128]
            top = np.abs(v).max()
            s = 127
            if top > 0:
                s = next((c for c in range(1, 255) if top <= E4M3_MAX * 2.0 ** (c - 127)), 254)
            y = np.minimum(np.abs(v) * 2.0 ** (127 - s), E4M3_MAX)
            hi = np.searchsorted(E4M3_GRID, y).clip(1, 126)
            lo = hi - 1
            dl, dh = y - E4M3_GRID[lo], E4M3_GRID[hi] - y
            c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
            c = np.where(y == 0, 0, c)
            codes[r, 128 * b:128 * b + 128] = c | np.where(np.signbit(v), 128, 0)
            sf[r, b] = s
    return codes, sf


def dequantize(codes, sf):
    """float64 values of a checkpoint (scales row-major [R, C/128])."""
    v = on.decode_e4m3(codes).astype(np.float64).reshape(sf.shape + (128,))
    return (v * 2.0 ** (sf.astype(np.float64) - 127)[..., None]).reshape(codes.shape)


# ------------------------------------------------------------ rows and tokens
def combine(D, rows, w=None):
    T, k = rows.shape
    out = np.zeros((T, D.shape[1]))
    for t in range(T):
        for j in range(k):
            if rows[t, j] >= 0:
                out[t] += (1.0 if w is None else float(w[t, j])) * D[rows[t, j]]
    return out


def combine_backward(dout, D, rows, w):
    """({row: gradient}, dw)."""
    T, k = rows.shape
    dD, dw = {}, np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if rows[t, j] >= 0:
                dD[int(rows[t, j])] = dout[t] * (1.0 if w is None else float(w[t, j]))
                dw[t, j] = dout[t] @ D[rows[t, j]]
    return dD, dw


def _sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def gate_up(h):
    b = h.reshape(h.shape[0], -1, 2, 128)
    return b[:, :, 0].reshape(h.shape[0], -1), b[:, :, 1].reshape(h.shape[0], -1)


def interleave(g, u):
    R = g.shape[0]
    return np.stack([g.reshape(R, -1, 128), u.reshape(R, -1, 128)], axis=2).reshape(R, -1)


def swiglu(h):
    g, u = gate_up(h)
    return g * _sigmoid(g) * u


def swiglu_backward(dy, h, w):
    """(dh, w * y, dw) of rows h [R, N] with routing weights w [R]."""
    g, u = gate_up(h)
    s = _sigmoid(g)
    y = g * s * u
    d = dy * w[:, None]
    return interleave(d * u * s * (1 + g * (1 - s)), d * g * s), y * w[:, None], (dy * y).sum(1)
