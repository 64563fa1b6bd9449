"""The experts' products where they can go wrong beyond the sizes and tables of
test_gpu_products: sums beyond fp32's largest number, the parts of fp32
operands, scratch that other calls use too."""
import pytest
import torch

import products_reference as ref
import swiglu_mlp_top_gb300 as mm
from test_gpu_products import on_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def beyond(exact):
    """fp32's value of sums, none of them near its largest number: those beyond it are infinities of their sign."""
    assert not bool(((exact.abs() >= 2.0 ** 127) & (exact.abs() < 2.0 ** 128)).any())
    return torch.where(exact.abs() >= 2.0 ** 128, torch.sign(exact) * torch.inf, exact)


def check_overflow(got, exact, terms, n, what):
    """Infinities where the definition's sums (of terms of one sign) are beyond fp32, else sums within
    the bound of products_reference."""
    got, want = got.cpu().double(), beyond(exact)
    far = want.isinf()
    assert not bool(got.isnan().any()), (what, int(got.isnan().sum()))
    assert torch.equal(got[far], want[far]), what
    ref.close_sum(torch.where(far, 0.0, got), torch.where(far, 0.0, want), torch.where(far, 0.0, terms), n, F32, what)


@pytest.mark.parametrize("rows,K,N", [
    (8, 96, 72), (20, 2432, 40),              # streamed
    (5, 97, 72),                              # few rows of an odd width
    (300, 96, 72), (300, 515, 130),           # tiles
    (300, 4096, 130)])                        # tiles, the sum in parts
@pytest.mark.parametrize("top", [75.0, 63.2])
def test_fp32_sums_that_overflow(rows, K, N, top):
    """Operands of one sign whose products (2^150) or whose sums alone
    (products of 2^126.4) are beyond fp32: infinities of the sums' sign, as
    fp32 products have them, and no NaN; other rows and columns are as ever."""
    gen = torch.Generator().manual_seed(rows + K)
    big = lambda *s: torch.exp2(top + torch.rand(*s, generator=gen) * (1.0 if top > 64 else 0.1))  # noqa: E731
    x, w, dy = big(rows, K), big(N, K), big(rows, N)
    x[1::2] *= -1                             # rows of the other sign
    dy[1::2] *= -1                            # ... so that the products that dw adds have one sign
    x[2::3] *= 2.0 ** -80                     # rows, and columns of the weights, of far smaller numbers
    dy[2::3] *= 2.0 ** -80
    w[1::3] *= 2.0 ** -80
    y = mm.grouped_matmul(x.cuda(), w.cuda())
    check_overflow(y, *ref.matmul(x, w, None, torch.zeros(rows, N)), K, "ys")
    dx, dw = mm.grouped_matmul_backward(dy.cuda(), x.cuda(), w.cuda())
    (wdx, tdx), (wdw, tdw) = ref.matmul_backward(dy, x, w, None, torch.zeros(rows, K))
    check_overflow(dx, wdx, tdx, N, "dxs")
    check_overflow(dw, wdw, tdw, rows, "dw")


@pytest.mark.parametrize("rows", [8, 300])
def test_fp32_overflow_stays_in_its_results(rows):
    """A result whose products overflow to both sides is not finite, and the others do not change by a bit."""
    gen = torch.Generator().manual_seed(rows)
    K, N = 264, 72
    x, w = torch.randn(rows, K, generator=gen), torch.randn(N, K, generator=gen)
    clean = mm.grouped_matmul(x.cuda(), w.cuda()).cpu()
    x[3] *= 2.0 ** 100
    w[7] *= 2.0 ** 80
    y = mm.grouped_matmul(x.cuda(), w.cuda()).cpu()
    # products of 2^180 of both signs: their sum, rounded once, is an infinity; added one by one in
    # fp32 they are inf - inf, a NaN; the tensor cores add sixteen products wider than fp32 before
    # they round, and keep the first infinity.  A finite number is none of these.
    assert not bool(y[3, 7].isfinite())
    keep = torch.ones(rows, N, dtype=torch.bool)
    keep[3], keep[:, 7] = False, False
    if rows > 40:                             # tiles: no result depends on its neighbours
        assert torch.equal(y[keep], clean[keep])
    want, terms = ref.matmul(x, w, None, torch.zeros(rows, N))
    ref.close_sum(torch.where(keep, y, 0.0), torch.where(keep, want, 0.0), torch.where(keep, terms, 0.0), K, F32, "ys")
