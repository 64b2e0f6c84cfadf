"""The error of routing scores that the header states, over the whole range of
logits, against float64.

In units of 2^-24, relative, for results above 2^-126:
  a sigmoid score 9; a softmax score |d| + E/16 + 26, d the logit's distance
  from the largest; renormalised weights 2 D + 26, D the largest |d| among the
  chosen (sigmoid: 0); one more for a scale other than 1.
They follow from the arithmetic: the hardware's 2^x is off by 4 units (two in the
last place) and its reciprocal by 2, an exponential with its correction by 5;
d itself is rounded, by |d|; a sum of E positive terms, at most E/16 + 1 of
them in a lane and five steps across, by E/16 + 5 beside its terms' mean error,
and the mean of |d| weighted by the scores is at most ln E < 7."""
import pytest
import torch

from moe_grouped_gemm_side_gb300 import binding as mb
from tests import ops_util as ou

pytestmark = pytest.mark.gpu

U, TINY = ou.U32, 2.0 ** -126


def run(x, k, score, renorm, bias=None, scale=1.0):
    T = x.shape[0]
    idx = torch.empty((T, k), dtype=torch.int32, device=x.device)
    w = torch.empty((T, k), device=x.device)
    mb.route(x, idx, w, score=score, renorm=renorm, bias=bias, scale=scale)
    return idx.long(), w.double()


def within(w, ref, units):
    err = (w - ref).abs()
    big = ref > 2 * TINY
    worst = (err / (ref * units * U))[big].max().item()
    assert worst <= 1.0, f"{worst:.2f} times the stated error"
    assert (w[~big] <= 4 * TINY).all()


def logits(seed, T, E, lo, hi, dtype, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return (lo + (hi - lo) * torch.rand(T, E, generator=g, device=device)).to(dtype)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,T", [(16, 60000), (64, 6000), (300, 500)])
def test_sigmoid_scores(E, T, dtype, bias, cuda):
    for lo, hi in ((-95.0, 95.0), (-4.0, 4.0), (-88.0, -80.0)):
        x = logits(E, T, E, lo, hi, dtype, cuda)
        x[0, :3] = torch.tensor([-3e38, 3e38, -1000.0])
        b = torch.zeros(E, device=cuda) if bias else None
        idx, w = run(x, min(E, 32), "sigmoid", False, b)
        within(w, torch.special.expit(x.double().gather(1, idx)), 9.0)
        idx, w = run(x, min(E, 32), "sigmoid", True, b, 2.5)
        s = torch.special.expit(x.double().gather(1, idx))
        keep = s.max(1).values > TINY * 2.0 ** 24            # all of a row may be flushed
        if keep.any():
            within(w[keep], (2.5 * s / s.sum(1, keepdim=True))[keep], 27.0)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,T", [(16, 60000), (64, 6000), (256, 20011), (1000, 500)])
def test_softmax_scores(E, T, dtype, bias, cuda):
    k = min(E, 32)
    b = torch.zeros(E, device=cuda) if bias else None
    for lo, hi in ((-80.0, 0.0), (-3.0, 3.0), (1000.0, 1060.0)):
        x = logits(E + 1, T, E, lo, hi, dtype, cuda)
        v = x.double()
        d = v.max(1, keepdim=True).values - v
        p = torch.softmax(v, 1)
        idx, w = run(x, k, "softmax", False, b)
        within(w, p.gather(1, idx), d.gather(1, idx) + E / 16 + 26)
        idx, w = run(x, k, "softmax", True, b, 2.5)
        s, D = p.gather(1, idx), d.gather(1, idx).max(1, keepdim=True).values
        within(w, 2.5 * s / s.sum(1, keepdim=True), (2 * D + 27).expand_as(s))


def test_one_expert_far_above_many_equal_ones(cuda):
    """The error of the sum does not vanish with d: 1023 equal terms carry one
    rounding of their argument, and add up."""
    d = torch.linspace(-12.0, -2.0, 4001, device=cuda)
    d[0] = -5.5987344
    x = d[:, None].repeat(1, 1024)
    x[:, 700] = 0.0
    idx, w = run(x, 2, "softmax", False)
    assert (idx[:, 0] == 700).all() and (idx[:, 1] == 0).all()
    v = x.double()
    p = torch.softmax(v, 1).gather(1, idx)
    within(w, p, (v.max(1, keepdim=True).values - v).gather(1, idx) + 1024 / 16 + 26)
