"""The workloads of perf/operators.py: the library's calls against the plain
form on small cases of every operator, layout and type, whole buffers at a
time (rows that no choice fills stay as they were in both)."""
import importlib.util
import os

import pytest
import torch

from tests import ops_util as ou

pytestmark = pytest.mark.gpu

_AT = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")


def workloads(own):
    spec = importlib.util.spec_from_file_location(f"operator_workloads_{own}", _AT)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.own = own
    return m


def routes():
    for op in ("route", "route_bwd"):
        for logits in ("bf16", "f32"):
            for score, bias, groups, top, renorm in (("softmax", False, 1, 1, True), ("softmax", False, 4, 1, False),
                                                     ("sigmoid", True, 4, 2, True), ("softmax", True, 1, 1, False),
                                                     ("sigmoid", False, 1, 1, False)):
                yield dict(op=op, T=37, unused=4, E=96, k=6, score=score, groups=groups, top_groups=max(1, groups // 2),
                           group_top=top, bias=bias, renorm=renorm, scale=2.5, logits=logits)


def layouts():
    yield dict(layout="masked", align=0, m_max=48)
    yield dict(layout="contiguous", align=16, m_max=0)


def cases():
    yield from routes()
    for at in layouts():
        for src, dst in (("bf16", "bf16"), ("bf16", "e4m3"), ("e4m3", "bf16"), ("e4m3", "e4m3")):
            for ckpt in ((False, True) if src == "bf16" else (False,)):
                yield dict(op="dispatch", T=41, unused=5, E=5, k=3, K=384, src=src, dst=dst, ckpt=ckpt, **at)
        for weights in (True, False):
            yield dict(op="combine", T=41, unused=5, E=5, k=3, K=384, weights=weights, **at)
        yield dict(op="combine_bwd", T=41, unused=5, E=5, k=3, K=384, **at)
        for out in ("bf16", "e4m3"):
            for N in (256, 768):
                yield dict(op="swiglu_save", T=41, unused=0, E=5, k=3, N=N, out=out, **at)
        yield dict(op="swiglu_bwd", T=41, unused=0, E=5, k=3, N=768, **at)


def rows_of(c, codes, scales):
    """Codes [.., C] and their scales as float64 rows."""
    G = scales.shape[-1]
    v = codes.double().view(-1, codes.shape[-1])
    s = scales.double().view(-1, v.shape[1] // 128, G).transpose(1, 2).reshape(v.shape[0], -1)
    return v * s.repeat_interleave(128, 1), s.repeat_interleave(128, 1)


@pytest.mark.parametrize("case", list(cases()), ids=lambda c: "-".join(str(v) for v in c.values()))
def test_calls_against_the_plain_form(case, cuda):
    plain, own = workloads(False), workloads(True)
    want = plain.run(plain.prepare(case, 77))
    state = own.prepare(case, 77)
    got = own.run(state)
    assert state["status"].item() == 0 and want.keys() == got.keys()
    if case["op"] == "swiglu_save" and case["out"] == "e4m3":
        # y differs in its last fp32 bits, so a code may fall on the next value:
        # 2^-3 of it apart at most (2^-9 of the scale among the subnormals)
        (a, s), (b, r) = rows_of(case, got.pop("Y"), got.pop("SFY")), rows_of(case, want.pop("Y"), want.pop("SFY"))
        assert ((a - b).abs() <= 2.0 ** -3 * b.abs() + 2.0 ** -9 * torch.maximum(s, r)).all()
    for name, w in want.items():
        g = got[name]
        assert g.dtype == w.dtype and g.shape == w.shape, name
        if w.dtype == torch.int32 or w.element_size() == 1:            # maps, codes and scales
            assert torch.equal(g.view(torch.uint8), w.view(torch.uint8)), name
        elif w.dtype == torch.bfloat16:
            # both round once, of fp32 values a few rounding units apart: one step
            # of the type at most, and terms that cancel to the sum's size
            top = w.double().abs().max().item()
            assert ((g.double() - w.double()).abs() <= 2 * ou.BF16 * w.double().abs() + 2.0 ** -14 * top).all(), name
        else:
            # sums of 384 terms in two orders: 384 rounding units of the terms'
            # magnitudes, some four times the largest sum
            top = w.double().abs().max().item()
            assert ((g.double() - w.double()).abs() <= 2.0 ** -12 * top).all(), name
