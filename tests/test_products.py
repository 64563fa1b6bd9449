"""The experts' products without a GPU: the C entry points and the Python
calls refuse what they cannot do before anything is launched, and the 64-bit
forms that the GPU tests compare with hold against differences."""
import ctypes as C

import pytest
import torch

import products_reference as ref
import swiglu_mlp_top_gb300 as mm
from swiglu_mlp_top_gb300 import _lib as L

F = C.c_void_p(1 << 20)           # never dereferenced: validation fails first
ODD = C.c_void_p((1 << 20) + 2)
BF, F32 = L.MM_DTYPE_BF16, L.MM_DTYPE_F32
BAD, UNS, WS, OK = L.MM_ERR_INVALID_ARG, L.MM_ERR_UNSUPPORTED, L.MM_ERR_WORKSPACE, L.MM_OK
FAR = L.MM_GROUPED_MAX_DIM + 1


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return L.load()


def test_forward_refusals(lib):
    def call(xs=F, w=F, off=F, cnt=F, rows=10, K=64, N=64, E=4, dt=BF, ys=F, ws=F, wsb=1 << 34, status=F):
        return lib.mm_grouped_matmul(xs, w, off, cnt, rows, K, N, E, dt, ys, ws, wsb, status, None)
    for kw in (dict(dt=7), dict(rows=-1), dict(K=0), dict(N=0), dict(E=0), dict(xs=None), dict(xs=ODD), dict(w=None), dict(w=ODD),
               dict(ys=None), dict(ys=ODD), dict(off=None), dict(cnt=None), dict(off=None, cnt=None), dict(off=ODD), dict(cnt=ODD),
               dict(status=ODD)):
        assert call(**kw) == BAD, kw
    for kw in (dict(E=65), dict(K=FAR), dict(N=FAR), dict(rows=L.MM_GROUPED_MAX_ROWS + 1)):
        assert call(**kw) == UNS, kw
    assert call(rows=0, xs=None, ys=None) == OK
    need = lib.mm_grouped_matmul_workspace_bytes(10, 65, 64, 4, BF)
    if need:
        assert call(K=65, wsb=need - 1) == WS and call(K=65, ws=None) == WS and call(K=65, ws=ODD) == WS
    assert lib.mm_grouped_matmul_workspace_bytes(10, 64, 64, 4, BF) == 0
    for bad in ((10, 64, 64, 4, 7), (-1, 64, 64, 4, BF), (10, 0, 64, 4, BF), (10, 64, 64, 65, BF), (10, FAR, 64, 4, BF)):
        assert lib.mm_grouped_matmul_workspace_bytes(*bad) == 0


def test_backward_refusals(lib):
    def call(dys=F, xs=F, w=F, off=F, cnt=F, rows=10, K=64, N=64, E=4, dt=BF, dxs=F, dw=F, ws=F, wsb=1 << 34, status=F):
        return lib.mm_grouped_matmul_backward(dys, xs, w, off, cnt, rows, K, N, E, dt, dxs, dw, ws, wsb, status, None)
    for kw in (dict(dt=7), dict(rows=-1), dict(K=0), dict(N=0), dict(E=0), dict(dys=None), dict(dys=ODD), dict(xs=None), dict(xs=ODD),
               dict(w=None), dict(w=ODD), dict(dxs=ODD), dict(dw=ODD), dict(dxs=None, dw=None), dict(off=None), dict(cnt=None),
               dict(off=None, cnt=None), dict(cnt=ODD), dict(status=ODD), dict(rows=0, dw=ODD)):
        assert call(**kw) == BAD, kw
    for kw in (dict(E=65), dict(K=FAR), dict(N=FAR), dict(rows=L.MM_GROUPED_MAX_ROWS + 1)):
        assert call(**kw) == UNS, kw
    assert call(rows=0, dw=None) == OK
    need = lib.mm_grouped_matmul_backward_workspace_bytes(10, 65, 64, 4, BF)
    if need:
        assert call(K=65, wsb=need - 1) == WS and call(K=65, ws=None) == WS
    assert lib.mm_grouped_matmul_backward_workspace_bytes(10, 64, 64, 65, BF) == 0


def test_mx4_refusals(lib):
    for fn, order in ((lib.mm_mx4_quantize, lambda x, c, e, R, C, dt, n: (x, R, C, dt, n, c, e, None)),
                      (lib.mm_mx4_dequantize, lambda x, c, e, R, C, dt, n: (c, e, R, C, dt, n, x, None))):
        def call(x=F, c=F, e=F, R=4, C=64, dt=BF, n=F):
            return fn(*order(x, c, e, R, C, dt, n))
        for kw in (dict(dt=7), dict(R=-1), dict(C=0), dict(x=None), dict(c=None), dict(e=None), dict(x=ODD), dict(c=ODD), dict(e=ODD), dict(n=ODD)):
            assert call(**kw) == BAD, kw
        assert call(C=FAR) == UNS and call(R=1 << 31) == UNS and call(R=0, x=None) == OK

    def call(x=F, xe=F, wc=F, we=F, off=F, cnt=F, rows=10, K=64, N=64, E=4, ys=F, ws=F, wsb=1 << 34, status=F):
        return lib.mm_mx4_matmul(x, xe, wc, we, off, cnt, rows, K, N, E, ys, ws, wsb, status, None)
    for kw in (dict(rows=-1), dict(K=0), dict(N=0), dict(E=0), dict(x=None), dict(x=ODD), dict(xe=ODD), dict(wc=None), dict(we=None),
               dict(we=ODD), dict(ys=None), dict(ys=ODD), dict(off=None), dict(cnt=None), dict(off=None, cnt=None), dict(off=ODD), dict(status=ODD)):
        assert call(**kw) == BAD, kw
    for kw in (dict(E=65), dict(K=FAR), dict(N=FAR), dict(rows=L.MM_GROUPED_MAX_ROWS + 1)):
        assert call(**kw) == UNS, kw
    assert call(rows=0, x=None, ys=None) == OK
    for xe, four in ((F, 1), (None, 0)):
        need = lib.mm_mx4_matmul_workspace_bytes(4000, 64, 64, 4, four)
        if need:
            assert call(rows=4000, xe=xe, wsb=need - 1) == WS and call(rows=4000, xe=xe, ws=None) == WS
    assert lib.mm_mx4_matmul_workspace_bytes(10, 64, 64, 65, 1) == 0


def test_python_calls_refuse_what_is_not_on_the_gpu():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    q = {"codes": torch.zeros(4, 32, dtype=torch.uint8), "exps": torch.zeros(1, 4, 4, dtype=torch.uint8), "cols": 64}
    for call in (lambda: mm.grouped_matmul(x, w), lambda: mm.grouped_matmul_backward(x, x, w), lambda: mm.mx4_quantize(x),
                 lambda: mm.mx4_dequantize(q), lambda: mm.mx4_matmul(x, q), lambda: mm.mx4_matmul(q, q)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


# ---------------------------------- the 64-bit forms against differences
D = 2.0 ** -10


@pytest.mark.parametrize("plan", [None, ref.tables([3, 0, 5, 1], align=4, start=2)])
def test_gradient_against_differences(plan):
    """The product is linear in each operand, so a central difference is off by
    its own roundings alone: 2^-52 of the loss's terms over D."""
    gen = torch.Generator().manual_seed(0)
    rand = lambda *shape: torch.randn(*shape, generator=gen, dtype=torch.float64)  # noqa: E731
    R, K, N = 24, 7, 5
    x, w, dy = rand(R, K), rand(*([4] if plan else []), N, K), rand(R, N)
    inside = torch.zeros(R, 1, dtype=torch.float64)
    for _, a, b, _ in ref.spans(plan, R):
        inside[a:b] = 1

    def loss(x, w):
        y, terms = ref.matmul(x, w, plan, torch.zeros(R, N))
        return (y * dy * inside).sum(), (terms * dy.abs()).sum()

    (dx, _), (dw, _) = ref.matmul_backward(dy, x, w, plan, torch.zeros(R, K))
    dx = dx * inside
    size = loss(x, w)[1]
    for way, got, at in ((rand(*x.shape), dx, lambda h, v: loss(x + h * v, w)), (rand(*w.shape), dw, lambda h, v: loss(x, w + h * v))):
        slope = (at(D, way)[0] - at(-D, way)[0]) / (2 * D)
        assert abs(slope - (got * way).sum()) <= 64 * (K + R * N) * 2.0 ** -52 / D * size


def test_e2m1_codes_are_the_formats():
    """Sign, two exponent bits of bias 1 and one fraction bit, subnormal below 1."""
    for c in range(8):
        e, f = c >> 1, c & 1
        assert ref.E2M1[c] == (f / 2 if e == 0 else (1 + f / 2) * 2.0 ** (e - 1))
    v = torch.arange(0, 6.0, 2.0 ** -6, dtype=torch.float64)
    code = ref.nearest_e2m1(v)
    dist = (v[:, None] - ref.E2M1[None]).abs()
    assert torch.equal(dist.gather(1, code[:, None])[:, 0], dist.amin(1))
    ties = (dist == dist.amin(1, keepdim=True)).sum(1) == 2
    assert int(ties.sum()) == 7 and bool((code[ties] % 2 == 0).all())


def test_quantised_values_are_near():
    x = torch.randn(40, 100, generator=torch.Generator().manual_seed(3))
    _, exps, values = ref.quantise(x)
    scale = torch.exp2(exps.permute(1, 0, 2).reshape(40, -1)[:, :4].double() - 127).repeat_interleave(32, 1)[:, :100]
    bound = torch.maximum(x.double().abs() / 4, scale / 4)
    assert bool(((values - x.double()).abs() <= bound).all())
