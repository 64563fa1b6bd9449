"""The order in which the kernels' sources wait for their predecessor and let
their successor launch (programmatic dependent launch), read from the sources:
a violation is a race that no run has to show.  Lexical order is execution
order: both stand in straight-line code, but for the grouped GEMM, where a
later down slot triggers at once and its epilogue waits.  That slot's
successor is the next slot, whose early loads were complete before the first
one, or the next call's first kernel, which loads nothing early."""
import os
import re

import pytest

from swiglu_mlp_top_gb300 import build

WAIT = re.compile(r'asm volatile\("griddepcontrol\.wait|pdl_enter\(\);')
TRIGGER = re.compile(r'asm volatile\("griddepcontrol\.launch_dependents|pdl_enter\(\);')


def kernels():
    """(name, body) of every kernel of the library."""
    out = []
    for path in build._sources():
        with open(path) as f:
            text = f.read()
        for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", text):
            i = text.index("{", m.end())
            depth, j = 1, i + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[j], 0)
                j += 1
            out.append((f"{os.path.basename(path)}:{m.group(1)}", text[i:j]))
    return out


KERNELS = kernels()


def test_the_kernels_are_found():
    names = [n for n, _ in KERNELS]
    for want in ("routing.cu:router_tc_kernel", "routing.cu:dispatch_kernel", "decode_sw.cu:decode_sw_kernel",
                 "gemm_tc.cu:grouped_gemm_kernel", "block_norm.cu:block_norm_ring_kernel", "permute.cu:permute_kernel"):
        assert want in names


@pytest.mark.parametrize("name,body", [pytest.param(n, b, id=n) for n, b in KERNELS if WAIT.search(b)])
def test_a_successor_launches_only_behind_the_wait(name, body):
    """Else a successor that reads something before its own wait, relying on
    the kernels before its predecessor, would read what those still write."""
    trigger = TRIGGER.search(body)
    assert trigger is None or WAIT.search(body).start() <= trigger.start(), name


LOAD = r"tma_load|tma_gather|row_load|\bcp\.async\.(?!bulk\.prefetch)"


def straight_line(body):
    """The body without comments and lambdas, and {name: body} of those: what a
    lambda does happens where it is called."""
    code, lambdas = re.sub(r"//[^\n]*", "", body), {}
    while True:
        m = re.search(r"auto (\w+) = \[[^]]*\]\([^)]*\)[^{;]*\{", code)
        if m is None:
            return code, lambdas
        depth, j = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(code[j], 0)
            j += 1
        lambdas[m.group(1)] = code[m.end():j]
        code = code[:m.start()] + code[j:]


@pytest.mark.parametrize("name,body", [pytest.param(n, b, id=n) for n, b in KERNELS
                                       if WAIT.search(b) and n != "routing.cu:dispatch_kernel"])
def test_nothing_is_loaded_before_the_wait(name, body):
    """What a kernel reads may be its predecessor's output, a weight as well as
    an activation.  The dispatch alone copies rows of x first: its predecessor
    is always the router, which lets it launch only behind its own wait.  (A
    prefetch into L2 reads nothing.)"""
    code, lambdas = straight_line(body)
    loaders = [n for n, b in lambdas.items() if re.search(LOAD, b)]
    load = re.search("|".join([LOAD] + [rf"\b{n}\(" for n in loaders]), code)
    assert load is None or WAIT.search(code).start() < load.start(), (name, load.group())
