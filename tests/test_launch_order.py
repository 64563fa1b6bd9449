"""The order in which the kernels' sources wait for their predecessor and let
their successor launch (programmatic dependent launch), read from the sources:
a violation is a race that no run has to show.  Lexical order is execution
order here: in every kernel both stand in straight-line code."""
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
