"""Rules that the operators' CUDA sources keep and that no run shows: what a
kernel that overlaps the one before it reads, and state that host threads
share.  Reads the sources only; runs on the CPU."""
import os
import re

import pytest

pytestmark = pytest.mark.cpu

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_grouped_gemm_side_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return re.sub(r"__launch_bounds__\((?:[^()]|\([^()]*\))*\)", "", text)


def sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h")))


def bodies(text):
    """Name and body of every function defined at the outermost level of a file
    (namespaces aside)."""
    for m in re.finditer(r"\n(?:template[^\n]*\n)?(?:__global__|__device__|static|inline)[^;{]*?(\w+)\(([^;{]*)\)\s*(?:const\s*)?{",
                         text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield m.group(1), text[m.end():at]


def test_overlapped_kernels_read_coherently():
    """A kernel that is launched while the one before it runs may read what that
    one writes after griddepcontrol.wait, and not by the non-coherent path
    (__ldg, ld.global.nc), which is for data that nothing writes as long as the
    kernel is there.  Functions that it calls after the wait are held to the
    same."""
    seen = 0
    for name in sources():
        text = source(name)
        funcs = dict(bodies(text))
        for fn, body in funcs.items():
            if "griddepcontrol.wait" not in body:
                continue
            seen += 1
            after = body.split("griddepcontrol.wait", 1)[1]
            reads = [after] + [funcs[f] for f in set(re.findall(r"\b(\w+)(?:<[^<>;]*>)?\(", after)) if f in funcs]
            for text_after in reads:
                assert "__ldg(" not in text_after and "global.nc" not in text_after, (name, fn)
    assert seen >= 2


def test_state_of_host_threads_is_atomic():
    """What a launch remembers between calls may be written by several host
    threads at once: every mutable static of the operators and of what they call is
    an atomic.  (The GEMMs' per-device flags only ever go from false to true.)"""
    for name in sources():
        if name in ("gemm_fwd.cu", "gemm_kgrouped.cu"):
            continue
        for line in re.findall(r"^\s*static\s[^\n(]*[;={][^\n]*$", source(name), re.M):
            if not re.match(r"\s*static\s+(const\b|constexpr\b)", line):
                assert re.match(r"\s*static\s+std::atomic<", line), (name, line)
