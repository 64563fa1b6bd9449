"""The C entries when host memory runs out: no C++ exception leaves them (one
would end the calling process).  A child process runs with an operator new that
throws on this thread while a flag is set; the flag covers one C call at a time
and the GPU sees ordinary work only."""
import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

NEW = """
#include <cstdlib>
#include <new>
static thread_local int failing = 0, asked = 0;
extern "C" int fail_new(int on) { int n = asked; failing = on; asked = 0; return n; }
void* operator new(std::size_t n) {
  if (failing) { ++asked; throw std::bad_alloc(); }
  void* p = std::malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  return p;
}
void* operator new(std::size_t n, std::align_val_t a) {
  if (failing) { ++asked; throw std::bad_alloc(); }
  const std::size_t al = static_cast<std::size_t>(a);
  void* p = std::aligned_alloc(al, (n + al - 1) / al * al);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p, std::align_val_t) noexcept { std::free(p); }
void operator delete(void* p, std::size_t, std::align_val_t) noexcept { std::free(p); }
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
"""

CHILD = """
import ctypes as C, sys
import torch
import swiglu_mlp_top_gb300 as mm
from swiglu_mlp_top_gb300 import _lib as L

fail_new = C.CDLL(sys.argv[1]).fail_new
lib = L.load()
BF = torch.bfloat16
E, k, coef = 4, 2, 0.01
rand = lambda *s, std=1.0: (std * torch.randn(*s, device="cuda")).to(BF)
H, I = 256, 192
W = lambda: [[rand(*s, std=0.05) for s in ((I, H), (I, H), (H, I))] for _ in range(E)]


def without_memory(call):
    '''call() with no host memory for C++ objects: its result and how often memory was asked for.'''
    torch.cuda.synchronize()
    fail_new(1)
    try:
        rc = call()
    finally:
        asked = fail_new(0)
    torch.cuda.synchronize()
    return rc, asked


# kernels loaded and their attributes set, then operands at addresses that no
# tensor map is kept for
def ffn(T, w, path, x, y, ws):
    return lib.mm_swiglu_ffn_ex(x.data_ptr(), *(t.data_ptr() for t in w), y.data_ptr(), T, H, I, L.MM_DTYPE_BF16,
                                ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream, path)


total = 0
for T in (16, 300, 1000):                    # the streaming kernel, the GEMMs
    ws = mm.new_workspace(mm.ffn_workspace_bytes(T, H, I, BF))
    old = W()[0]
    y0 = mm.swiglu_ffn(rand(T, H), *old, workspace=ws)
    x, w = rand(T, H), W()[0]
    ys = [torch.zeros(T, H, dtype=BF, device="cuda") for _ in range(2)]
    for y in ys:                             # what was not kept is made again
        rc, asked = without_memory(lambda: ffn(T, w, 0, x, y, ws))
        assert rc == L.MM_OK and asked > 0, (T, rc, asked)
        total += asked
    want = mm.swiglu_ffn(x, *w)
    assert all(torch.equal(y, want) for y in ys)

# a table of kernel attributes that cannot grow: refused with a code, and right afterwards
x, f = rand(300, 4096), rand(300, 4096)
r, n = torch.empty_like(x), torch.empty_like(x)
weight = torch.ones(4096, dtype=BF, device="cuda")
norm = lambda: lib.mm_block_norm(x.data_ptr(), f.data_ptr(), weight.data_ptr(), None, 0, weight.data_ptr(), 1.0, 1e-5, 300, 4096,
                                 L.MM_DTYPE_BF16, r.data_ptr(), n.data_ptr(), None, None, torch.cuda.current_stream().cuda_stream)
rc, asked = without_memory(norm)
assert rc == L.MM_ERR_CUDA and asked > 0, (rc, asked)
assert norm() == L.MM_OK
want = mm.block_norm(x, f, post_weight=weight, pre_weight=weight)
assert torch.equal(r, want[0]) and torch.equal(n, want[1])

# the launch hooks: a launch whose events cannot be kept goes untimed
lib.mm_profile_start(L.MM_KERNEL_NORM, 5)
rc, asked = without_memory(norm)
assert rc == L.MM_OK and asked > 0, (rc, asked)
assert norm() == L.MM_OK
ms, count = C.c_double(0), C.c_int(0)
assert lib.mm_profile_stop(C.byref(ms), C.byref(count)) == L.MM_OK and count.value == 1, count.value
print("asked", total)
"""


def test_no_exception_leaves_the_entries(tmp_path):
    import __graft_entry__
    __graft_entry__.build()
    src, lib, child = tmp_path / "new.cpp", tmp_path / "libnew.so", tmp_path / "child.py"
    src.write_text(NEW)
    child.write_text(textwrap.dedent(CHILD))
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    env = dict(os.environ, LD_PRELOAD=str(lib), PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, str(child), str(lib)], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
