"""Shared pieces of the tests of the operators around the grouped GEMMs.

Tolerances, derived from the arithmetic (u = 2^-24, the fp32 rounding unit):
* bf16 outputs round once: 8 significant bits, half a unit in the last place is
  at most 2^-8 |value|; on top of the fp32 error.
* fp32 sums of n products in any order: n u sum |products|.
* scores: exp and division to a few ulp; exp(x - max) also carries the
  rounding of x - max, |x - max| u; a sum of E of them (E + 2) u at most, in
  a tree far less.  SCORE_TOL(range, E) = (range + E + 64) u, relative.
* SwiGLU's fast exponential and division: (8 + 1.2 |g|) 2^-23, relative (the
  library's stated bound)."""
import numpy as np
import torch

U32 = 2.0 ** -24
BF16 = 2.0 ** -8


def score_tol(rng, E):
    return (rng + E + 64) * U32


def bf16_np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def np64(t):
    return t.detach().cpu().numpy().astype(np.float64)


def random_bf16(rng, shape, scale=1.0):
    """bf16 tensor on the CPU and its float64 values."""
    t = torch.from_numpy(rng.normal(size=shape).astype(np.float32) * np.float32(scale)).to(torch.bfloat16)
    return t, bf16_np(t)


def random_choices(rng, T, k, E, drop=0.15, skew=True):
    """int64 [T, k]: distinct experts per token, some tokens and choices at -1."""
    p = np.exp(rng.normal(size=E) * (1.0 if skew else 0.0))
    idx = np.stack([rng.choice(E, size=k, replace=k > E, p=p / p.sum()) for _ in range(T)]) if T else \
        np.zeros((0, k), dtype=np.int64)
    idx = idx.astype(np.int64)
    if T:
        idx[rng.random(T) < drop / 2] = -1
        idx[rng.random((T, k)) < drop / 2] = -1
    return idx


def i32(a, device):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(device)


def f32(a, device):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.float32)).to(device)


def status_word(device):
    return torch.zeros(1, dtype=torch.int32, device=device)
