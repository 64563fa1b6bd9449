"""The experts' products and 4-bit floating point against the 64-bit forms of
products_reference (bounds there).  Inputs of small whole numbers, whose sums
fp32 holds exactly, are compared exactly."""
import pytest
import torch

import products_reference as ref
import swiglu_mlp_top_gb300 as mm
from block_reference import close

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def groups(E, total, how, seed=0):
    """Sizes of E groups that add up to `total`."""
    gen = torch.Generator().manual_seed(31 * E + total + seed)
    if how == "one":
        return [0] * (E - 1) + [total]
    if how == "even":
        return [total // E + (e < total % E) for e in range(E)]
    p = torch.rand(E, generator=gen) ** 3 + 1e-3
    p[torch.randint(E, (1,), generator=gen)] = 0 if E > 1 else 1       # one of them empty
    return torch.bincount(torch.multinomial(p, total, replacement=True, generator=gen), minlength=E).tolist() if total else [0] * E


def on_gpu(plan):
    return None if plan is None else {k: v.cuda() for k, v in plan.items()}


def make(rows, width, dtype, gen, whole, plan, junk=True):
    """Rows of a sorted tensor; NaN outside the assignments (no call may see them)."""
    x = torch.randint(-3, 4, (rows, width), generator=gen).to(dtype) if whole else torch.randn(rows, width, generator=gen).to(dtype)
    if junk and plan is not None:
        keep = torch.zeros(rows, dtype=torch.bool)
        for _, a, b, _ in ref.spans(plan, rows):
            keep[a:b] = True
        x[~keep] = torch.nan
    return x


def check(counts, align, K, N, dtype, whole, start=0, tail=3):
    plan = None if counts is None else ref.tables(counts, align, start)
    rows = tail if plan is None else int(plan["offsets"][-1]) + tail
    E = 1 if plan is None else len(counts)
    gen = torch.Generator().manual_seed(K * 7 + N + rows)
    x, dy = make(rows, K, dtype, gen, whole, plan), make(rows, N, dtype, gen, whole, plan)
    shape = (N, K) if plan is None else (E, N, K)
    w = torch.randint(-2, 3, shape, generator=gen).to(dtype) if whole else (torch.randn(*shape, generator=gen) * 0.1).to(dtype)
    gplan = on_gpu(plan)
    xg, wg, dyg = x.cuda(), w.cuda(), dy.cuda()
    status = mm.new_workspace(256)

    mark = torch.full((rows, N), 7.0, dtype=dtype)
    y = mm.grouped_matmul(xg, wg, gplan, out=mark.cuda(), status_workspace=status)
    want, terms = ref.matmul(x, w, plan, mark)
    mark = torch.full((rows, K), 7.0, dtype=dtype)
    dx, dw = mm.grouped_matmul_backward(dyg, xg, wg, gplan, out=mark.cuda(), dw=torch.full(shape, 7.0, device="cuda"), status_workspace=status)
    (wdx, tdx), (wdw, tdw) = ref.matmul_backward(dy, x, w, plan, mark)
    assert mm.check_status(status) == 0
    longest = max(counts) if counts else rows
    if whole:
        # every partial sum is a whole number below 2^24: fp32 holds it, and one rounding remains
        assert max(terms.max(), tdx.max(), tdw.max(), 7) < 2 ** 24
        assert torch.equal(y.cpu(), want.to(dtype)), "ys"
        assert torch.equal(dx.cpu(), wdx.to(dtype)), "dxs"
        assert torch.equal(dw.cpu(), wdw.float()), "dw"
    else:
        ref.close_sum(y, want, terms, K, dtype, "ys")
        ref.close_sum(dx, wdx, tdx, N, dtype, "dxs")
        ref.close_sum(dw, wdw, tdw, longest, F32, "dw")


SIZES = [
    # counts, align, K, N
    ([1], 1, 64, 64), ([1], 1, 8, 8), ([2, 0, 1], 1, 72, 40), ([0, 0, 0], 4, 64, 64), ([130], 1, 64, 256),
    ([5, 0, 300, 1, 17], 1, 128, 200), ([5, 0, 300, 1, 17], 64, 128, 264), ([129, 127, 128, 256], 1, 192, 512),
    ([257, 31, 64, 0], 16, 768, 320), ([33, 95], 1, 2432, 96), ([40, 90], 5, 96, 2432),
    # widths with no access wider than an element common to all rows, and ones between
    ([70, 3, 200], 1, 65, 33), ([70, 3, 200], 7, 1001, 129), ([300], 1, 1, 1), ([20, 150], 3, 130, 1), ([20, 150], 1, 1, 130),
    ([20, 150], 1, 36, 52), ([20, 150], 1, 50, 68), ([64, 64], 1, 100, 7), ([3, 140], 1, 264, 999),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("counts,align,K,N", SIZES)
def test_products(counts, align, K, N, dtype):
    check(counts, align, K, N, dtype, whole=True)
    check(counts, align, K, N, dtype, whole=False, start=align)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,total,align,K,N,how", [
    (64, 64, 1, 256, 128, "skewed"), (64, 700, 128, 128, 136, "skewed"), (8, 2000, 64, 768, 640, "skewed"), (8, 1500, 1, 200, 768, "one"),
    (16, 16, 1, 2432, 768, "even"), (3, 1, 1, 768, 4864, "skewed"), (64, 4000, 1, 64, 64, "even")])
def test_many_groups(E, total, align, K, N, how, dtype):
    check(groups(E, total, how), align, K, N, dtype, whole=False)


@pytest.mark.parametrize("counts,align", [
    # few rows, most of them one expert's: its rows are shared out over blocks
    ([32], 1), ([17], 1), ([0, 33], 1), ([25, 0, 18], 1), ([9, 33, 2], 2), ([66, 3, 0, 1, 0, 0, 0, 0], 1), ([50, 0, 0, 5, 0, 0, 0, 0], 8),
    # the same for fp32
    ([15], 1), ([0, 19], 1), ([9, 0, 14], 1), ([9, 0, 8], 4), ([40, 0, 0, 1, 0, 0, 0, 0], 1), ([17, 0, 0, 7, 0, 0, 0, 0], 16)])
def test_few_rows_of_one_expert(counts, align):
    for K, N in ((256, 40), (2432, 72), (8, 17), (4096, 16), (1001, 33), (36, 20)):
        for dtype in (BF, F32):
            check(counts, align, K, N, dtype, whole=True)
    for K in (264, 100, 65):
        check(counts, align, K, 100, BF, whole=False)
        check(counts, align, K, 100, F32, whole=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("counts,align,K,N", [
    # few tiles with a long sum: cut into parts
    ([300], 1, 4096, 130), ([300], 1, 130, 4096), ([270, 500], 16, 2050, 72), ([3000], 1, 72, 60), ([100, 4000], 1, 64, 136), ([0, 700], 3, 1030, 257),
    ([2500, 0], 1, 33, 65)])
def test_sums_in_parts(counts, align, K, N, dtype):
    check(counts, align, K, N, dtype, whole=True)
    check(counts, align, K, N, dtype, whole=False, start=align)


@pytest.mark.parametrize("counts", [[200, 150], [20, 15], [40, 3]])
def test_fp32_of_every_size(counts):
    """Values that bf16 parts cannot hold (infinities, NaN, above 2^127, below
    2^-100) anywhere among the operands: the results are those of fp32 products."""
    gen = torch.Generator().manual_seed(12)
    E, K, N = 2, 72, 40
    plan = ref.tables(counts, 8)
    rows = int(plan["offsets"][-1]) + 3
    gplan = on_gpu(plan)
    for what, value in (("x", torch.inf), ("x", torch.nan), ("w", -torch.inf), ("x", 1.9 * 2.0 ** 127), ("w", 2.0 ** -120), ("dy", torch.inf), ("dy", 2.0 ** -130)):
        x, dy, w = torch.randn(rows, K, generator=gen), torch.randn(rows, N, generator=gen), torch.randn(E, N, K, generator=gen)
        if value == 2.0 ** -120:
            w = w * value                        # all of them: fp32's accuracy is wanted there too
        elif value == 2.0 ** -130:
            dy = dy * value
        else:
            {"x": x, "w": w[0], "dy": dy}[what][5, 7] = value
            if value == 1.9 * 2.0 ** 127:
                w, dy = w / 64, dy / 64          # no sum overflows
        y = mm.grouped_matmul(x.cuda(), w.cuda(), gplan, out=torch.zeros(rows, N, device="cuda"))
        dx, dw = mm.grouped_matmul_backward(dy.cuda(), x.cuda(), w.cuda(), gplan, out=torch.zeros(rows, K, device="cuda"))
        want, terms = ref.matmul(x, w, plan, torch.zeros(rows, N))
        (wdx, tdx), (wdw, tdw) = ref.matmul_backward(dy, x, w, plan, torch.zeros(rows, K))
        for got, exact, size, n, name in ((y, want, terms, K, "ys"), (dx, wdx, tdx, N, "dxs"), (dw, wdw, tdw, 200, "dw")):
            got = got.cpu()
            fine = exact.abs() < 2.0 ** 127
            assert torch.equal(torch.isnan(got), torch.isnan(exact)), (what, value, name)
            assert bool((got[exact.abs() == torch.inf] == exact[exact.abs() == torch.inf].float()).all()), (what, value, name)
            # results near fp32's smallest have steps of 2^-149
            close(torch.where(fine, got.double(), 0.0), torch.where(fine, exact, 0.0),
                  torch.where(fine, 2.0 ** -24 * exact.abs() + 2 * (n + 1) * 2.0 ** -24 * size + n * 2.0 ** -149, 0.0), name)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,K,N", [(1, 768, 768), (7, 64, 1000), (200, 515, 130), (1000, 128, 256)])
def test_one_matrix_for_all_rows(rows, K, N, dtype):
    check(None, 1, K, N, dtype, whole=True, tail=rows)
    check(None, 1, K, N, dtype, whole=False, tail=rows)


def test_no_rows():
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(4, 32, 64, dtype=BF, device="cuda")
    plan = on_gpu(ref.tables([0] * 4))
    y = mm.grouped_matmul(x, w, plan)
    dx, dw = mm.grouped_matmul_backward(y, x, w, plan, dw=torch.ones(4, 32, 64, device="cuda"))
    assert y.shape == (0, 32) and dx.shape == (0, 64) and not dw.any()
    q = mm.mx4_quantize(x)
    assert mm.mx4_dequantize(q).shape == (0, 64)
    assert mm.mx4_matmul(q, mm.mx4_quantize(w), plan).shape == (0, 32)


@pytest.mark.parametrize("R", [200, 30])
@pytest.mark.parametrize("sx,sw", [(-40, -40), (-60, -50), (-60, -66), (60, 50)])
def test_fp32_of_every_magnitude(sx, sw, R):
    """Products far from 1, down to those below the smallest normal number,
    where a sum is off by that number's steps."""
    gen = torch.Generator().manual_seed(6)
    K, N = 96, 72
    x, w, dy = torch.randn(R, K, generator=gen) * 2.0 ** sx, torch.randn(N, K, generator=gen) * 2.0 ** sw, torch.randn(R, N, generator=gen) * 2.0 ** sw
    y, dw = mm.grouped_matmul(x.cuda(), w.cuda()), mm.grouped_matmul_backward(dy.cuda(), x.cuda(), None)[1]
    for got, a, b, n in ((y, x, w.T, K), (dw, dy.T, x, R)):
        want, terms = a.double() @ b.double(), a.double().abs() @ b.double().abs()
        # each of the at most six products and their sums: 2^-24 of the terms' sizes, or half of the smallest step
        bound = 2 * (n + 1) * (2.0 ** -24 * terms + 6 * 2.0 ** -150)
        assert bool(((got.double().cpu() - want).abs() <= bound).all())


def test_one_gradient_at_a_time():
    gen = torch.Generator().manual_seed(5)
    x, w, dy = (torch.randn(*s, generator=gen).to(BF).cuda() for s in ((50, 64), (3, 96, 64), (50, 96)))
    plan = on_gpu(ref.tables([20, 0, 30]))
    dx, dw = mm.grouped_matmul_backward(dy, x, w, plan)
    a, none = mm.grouped_matmul_backward(dy, None, w, plan)
    assert none is None and torch.equal(a, dx)
    none, b = mm.grouped_matmul_backward(dy, x, None, plan)
    assert none is None and torch.equal(b, dw)


def test_tables_that_point_outside():
    """Entries outside the tensor are taken as the nearest inside: nothing else is read or written."""
    x, w = torch.ones(40, 64, dtype=BF, device="cuda"), torch.ones(3, 32, 64, dtype=BF, device="cuda")
    for off, cnt in (([-50, 10, 2 ** 30, 2 ** 31 - 1], [2 ** 31 - 1] * 3), ([-2 ** 31, -5, 20, 60], [-1, 5, 2 ** 30]), ([30, 20, 10, 0], [4, 4, 4])):
        plan = {"offsets": torch.tensor(off, dtype=torch.int32, device="cuda"), "counts": torch.tensor(cnt, dtype=torch.int32, device="cuda")}
        y = mm.grouped_matmul(x, w, plan, out=torch.full((40, 32), 7.0, dtype=BF, device="cuda"))
        dx, dw = mm.grouped_matmul_backward(y, x, w, plan)
        torch.cuda.synchronize()
        assert bool(((y == 64) | (y == 7) | (y == 0)).all()) and dw.shape == (3, 32, 64)


def test_tables_that_point_outside_many_rows():
    """The same where tiles of rows are taken, and with weights in 4 bits."""
    R, K, N = 700, 72, 136
    x, w = torch.ones(R, K, dtype=BF, device="cuda"), torch.ones(3, N, K, dtype=BF, device="cuda")
    wq, xq = mm.mx4_quantize(w), mm.mx4_quantize(x)
    status = mm.new_workspace(256)
    for off, cnt in (([-50, 300, 2 ** 30, 2 ** 31 - 1], [2 ** 31 - 1] * 3), ([-2 ** 31, -5, 400, 701], [-1, 5, 2 ** 30]), ([600, 300, 10, 0], [4, 4, 4])):
        plan = {"offsets": torch.tensor(off, dtype=torch.int32, device="cuda"), "counts": torch.tensor(cnt, dtype=torch.int32, device="cuda")}
        for dtype in (BF, F32):
            y = mm.grouped_matmul(x.to(dtype), w.to(dtype), plan, out=torch.full((R, N), 7.0, dtype=dtype, device="cuda"), status_workspace=status)
            mm.grouped_matmul_backward(y, x.to(dtype), w.to(dtype), plan, status_workspace=status)
            assert bool(((y == K) | (y == 7) | (y == 0)).all())
        for xs in (x, xq):
            y = mm.mx4_matmul(xs, wq, plan, out=torch.full((R, N), 7.0, dtype=BF, device="cuda"), status_workspace=status)
            assert bool(((y == K) | (y == 7) | (y == 0)).all())
    assert mm.check_status(status) == 0


def test_refusals_on_the_device():
    x, w = torch.zeros(6, 64, dtype=BF, device="cuda"), torch.zeros(2, 32, 64, dtype=BF, device="cuda")
    plan = on_gpu(ref.tables([2, 4]))
    q, wq = mm.mx4_quantize(x), mm.mx4_quantize(w)
    for bad in (lambda: mm.grouped_matmul(x, w), lambda: mm.grouped_matmul(x, w[0], plan), lambda: mm.grouped_matmul(x, w.float(), plan),
                lambda: mm.grouped_matmul(x, w[:, :, :32].contiguous(), plan), lambda: mm.grouped_matmul(x, w.transpose(1, 2), plan),
                lambda: mm.grouped_matmul(x, w[:1], plan), lambda: mm.grouped_matmul(x, w, plan, out=x),
                lambda: mm.grouped_matmul(x, w, {"offsets": plan["offsets"], "counts": plan["counts"].long()}),
                lambda: mm.grouped_matmul(x, w, plan, status_workspace=torch.zeros(8, device="cuda")),
                lambda: mm.grouped_matmul_backward(x[:, :32].contiguous(), None, None, plan),
                lambda: mm.grouped_matmul_backward(x, x, w, plan), lambda: mm.grouped_matmul_backward(x[:, :32].contiguous(), x, None, plan, out=x),
                lambda: mm.grouped_matmul_backward(x[:, :32].contiguous(), None, w, plan, dw=w.float()),
                lambda: mm.mx4_quantize(x[0]), lambda: mm.mx4_quantize(x.half()), lambda: mm.mx4_quantize(x, out=wq),
                lambda: mm.mx4_quantize(x, rows=torch.zeros(1, device="cuda")), lambda: mm.mx4_dequantize(dict(q, cols=96)),
                lambda: mm.mx4_dequantize(q, torch.float16), lambda: mm.mx4_dequantize(dict(q, exps=q["exps"][:, :3])),
                lambda: mm.mx4_matmul(x.float(), wq, plan), lambda: mm.mx4_matmul(q, wq), lambda: mm.mx4_matmul(x, q, plan),
                lambda: mm.mx4_matmul(dict(q, cols=63), wq, plan), lambda: mm.mx4_matmul(q, wq, plan, out=x.float())):
        with pytest.raises(ValueError):
            bad()


# --------------------------------------------- microscaled 4-bit floating point
def quantised(x, **kw):
    """mx4_quantize of x and the definition's, compared; the values on the CPU."""
    q = mm.mx4_quantize(x.cuda(), **kw)
    codes, exps, values = ref.quantise(x.reshape(-1, x.shape[-1]))
    assert torch.equal(q["exps"].cpu(), exps) and torch.equal(q["codes"].cpu().view(codes.shape), codes) and q["cols"] == x.shape[-1]
    return q, values.view(x.shape)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 32), (3, 768), (2, 33), (5, 127), (7, 128), (4, 129), (64, 2432), (33, 1000), (17, 1001),
                                 (100, 66), (9, 1028), (1000, 40), (2, 20000), (257, 96)])
def test_quantise(R, C, dtype):
    gen = torch.Generator().manual_seed(R + C)
    spread = torch.exp2(torch.randint(-60, 60, (R, 1), generator=gen).float())
    q, values = quantised((torch.randn(R, C, generator=gen) * spread).to(dtype))
    for out in (BF, F32):
        assert torch.equal(mm.mx4_dequantize(q, out).cpu().double(), values)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantise_at_the_edges(dtype):
    top = torch.finfo(dtype).max
    x = torch.zeros(16, 96)
    x[0, :8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])        # ties
    x[1, :8] = -x[0, :8]
    x[2, 0], x[2, 1] = 6.0, 2.0 ** -20                                            # vanishes beside 6
    x[3, 40] = torch.finfo(dtype).tiny / 4                                        # subnormal
    x[4, 40] = top
    x[5, 40] = -top * 0.6
    x[6, 33] = torch.inf
    x[7, 33], x[7, 1] = torch.nan, 3.0
    x[8, 95] = -torch.inf
    x[9, :32] = 7.0                                                               # between 6 and 8
    x[10, :32], x[10, 32:64] = 6.001, 5.999
    x[11] = 2.0 ** -126
    x[12, :32] = 2.0 ** -124 * 1.5
    x[13, :32] = 2.0 ** -124 * 1.75
    x[14] = -0.0
    x[15, :3] = torch.tensor([2.0 ** -127, -(2.0 ** -127) * 1.5, 2.0 ** -129])    # subnormal, and not zero
    q, values = quantised(x.to(dtype))
    back = mm.mx4_dequantize(q, F32).cpu().double()
    same = torch.where(values.abs() >= 2.0 ** 128, torch.sign(values) * torch.inf, values)
    assert torch.equal(torch.isnan(back), torch.isnan(same))
    assert torch.equal(torch.nan_to_num(back, nan=0.0, posinf=1.0, neginf=-1.0), torch.nan_to_num(same, nan=0.0, posinf=1.0, neginf=-1.0))
    assert torch.equal(torch.isnan(back).all(1), torch.tensor([False] * 16)) and bool(torch.isnan(back[6, 32:64]).all())


def test_quantise_experts_and_some_rows():
    gen = torch.Generator().manual_seed(2)
    w = torch.randn(3, 50, 100, generator=gen).to(BF)
    q, _ = quantised(w)
    assert q["codes"].shape == (3, 50, 64) and q["exps"].shape == (1, 150, 4)
    x = torch.randn(40, 100, generator=gen).to(BF)
    rows = torch.tensor([13], dtype=torch.int32, device="cuda")
    mark = {"codes": torch.full((40, 64), 9, dtype=torch.uint8, device="cuda"), "exps": torch.full((1, 40, 4), 9, dtype=torch.uint8, device="cuda"), "cols": 100}
    got = mm.mx4_quantize(x.cuda(), rows=rows, out=mark)
    codes, exps, values = ref.quantise(x)
    assert got is mark and torch.equal(got["codes"][:13].cpu(), codes[:13]) and torch.equal(got["exps"][:, :13].cpu(), exps[:, :13])
    assert bool((got["codes"][13:] == 9).all()) and bool((got["exps"][:, 13:] == 9).all())
    y = mm.mx4_dequantize(got, F32, rows=rows, out=torch.full((40, 100), 7.0, device="cuda"))
    assert torch.equal(y[:13].cpu().double(), values[:13]) and bool((y[13:] == 7).all())
    for n in (-3, 0, 41, 2 ** 31 - 1):                       # the nearest row inside
        y = mm.mx4_dequantize(mm.mx4_quantize(x.cuda()), F32, rows=torch.tensor([n], dtype=torch.int32, device="cuda"), out=torch.full((40, 100), 7.0, device="cuda"))
        assert torch.equal(y.cpu().double(), values if n > 40 else torch.full_like(values, 7.0))


MX_SIZES = [
    ([1], 1, 64, 64), ([1], 1, 32, 8), ([2, 0, 1], 1, 72, 40), ([0, 0, 0], 4, 64, 64), ([130], 1, 256, 192),
    ([5, 0, 300, 1, 17], 1, 128, 200), ([5, 0, 300, 1, 17], 64, 384, 264), ([129, 127, 128, 256], 1, 192, 512),
    ([257, 31, 64, 0], 16, 768, 320), ([33, 95], 1, 2432, 96), ([40, 90], 5, 96, 2432), ([70, 3, 200], 1, 65, 33),
    ([70, 3, 200], 7, 1001, 129), ([20, 150], 3, 130, 1), ([20, 150], 1, 1, 130), ([3, 9, 16, 8], 1, 768, 1216), ([64, 64], 1, 100, 7),
    ([1000, 600], 128, 1280, 576),
]


def check_mx4(counts, align, K, N, four, whole, tail=3):
    plan = None if counts is None else ref.tables(counts, align, 2)
    rows = tail if plan is None else int(plan["offsets"][-1]) + tail
    gen = torch.Generator().manual_seed(K * 5 + N + rows)
    shape = (N, K) if plan is None else (len(counts), N, K)
    if whole:
        # e2m1 values times powers of two near 1: the sums are multiples of 2^-4, exact in fp32
        pick = lambda *s: ref.E2M1[torch.randint(0, 6, s, generator=gen)] * torch.randint(-1, 2, s, generator=gen)  # noqa: E731
        x, w = pick(rows, K).to(BF), pick(*shape).to(BF)
    else:
        x, w = torch.randn(rows, K, generator=gen).to(BF), (torch.randn(*shape, generator=gen) * 0.1).to(BF)
    keep = torch.zeros(rows, dtype=torch.bool)
    for _, a, b, _ in ref.spans(plan, rows):
        keep[a:b] = True
    x[~keep] = torch.nan
    wq = mm.mx4_quantize(w.cuda())
    wv = ref.stored(w)[1]
    xg, xv = x.cuda(), x
    if four:
        xg, xv = mm.mx4_quantize(x.cuda()), ref.stored(x)[1]
    status = mm.new_workspace(256)
    mark = torch.full((rows, N), 7.0, dtype=BF)
    y = mm.mx4_matmul(xg, wq, on_gpu(plan), out=mark.cuda(), status_workspace=status)
    assert mm.check_status(status) == 0
    want, terms = ref.matmul(xv, wv, plan, mark)
    if whole:
        assert terms.max() < 2 ** 20
        assert torch.equal(y.cpu(), want.to(BF))
    else:
        ref.close_sum(y, want, terms, K, BF, "ys")


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("counts,align,K,N", MX_SIZES)
def test_mx4_products(counts, align, K, N, four):
    check_mx4(counts, align, K, N, four, whole=True)
    check_mx4(counts, align, K, N, four, whole=False)


@pytest.mark.parametrize("counts,align", [
    # few bf16 rows, most of them one expert's
    ([75], 1), ([33], 1), ([49, 40], 1), ([90, 0, 16], 1), ([65, 0, 9], 16), ([150, 9, 24, 0, 0, 0, 0, 0], 1), ([97, 0, 0, 2, 0, 0, 0, 0], 32)])
def test_mx4_few_rows_of_one_expert(counts, align):
    for K, N in ((256, 40), (2432, 72), (8, 17), (4096, 16)):
        check_mx4(counts, align, K, N, False, whole=True)
    check_mx4(counts, align, 264, 100, False, whole=False)


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("rows,K,N", [(1, 768, 768), (9, 64, 1000), (200, 515, 130), (700, 1024, 256)])
def test_mx4_one_matrix(rows, K, N, four):
    check_mx4(None, 1, K, N, four, whole=True, tail=rows)
    check_mx4(None, 1, K, N, four, whole=False, tail=rows)


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("rows", [4, 300])
def test_mx4_scales_of_every_size(rows, four):
    """Groups' scales over the whole range of the byte, alternating so that the products stay in fp32."""
    K, N = 256, 40
    gen = torch.Generator().manual_seed(rows)
    up = torch.exp2(torch.arange(K // 32).float() * 30 - 110).repeat_interleave(32)
    x, w = (torch.randn(rows, K, generator=gen) * up).to(BF), (torch.randn(N, K, generator=gen) / up).to(BF)
    wq, wv = mm.mx4_quantize(w.cuda()), ref.stored(w)[1]
    xg, xv = (mm.mx4_quantize(x.cuda()), ref.stored(x)[1]) if four else (x.cuda(), x)
    want, terms = ref.matmul(xv, wv, None, torch.zeros(rows, N))
    ref.close_sum(mm.mx4_matmul(xg, wq), want, terms, K, BF, "ys")


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("rows", [3, 200])
def test_mx4_nan_stays_in_its_rows(rows, four):
    """A group with a NaN or an infinity makes its row (of x) or its column (of w) NaN and nothing else."""
    K, N = 200, 70
    gen = torch.Generator().manual_seed(rows)
    x, w = torch.randn(rows, K, generator=gen).to(BF), torch.randn(N, K, generator=gen).to(BF)
    clean = mm.mx4_matmul(mm.mx4_quantize(x.cuda()) if four else x.cuda(), mm.mx4_quantize(w.cuda()))
    x[1, 5], w[11, 150] = torch.nan, torch.inf
    y = mm.mx4_matmul(mm.mx4_quantize(x.cuda()) if four else x.cuda(), mm.mx4_quantize(w.cuda()))
    bad = torch.zeros(rows, N, dtype=torch.bool)
    bad[1], bad[:, 11] = True, True
    assert torch.equal(torch.isnan(y).cpu(), bad) and torch.equal(y.cpu()[~bad], clean.cpu()[~bad])


# ---------------------------------------------------------- as they are used
def layer(T, H, I, E, k, align, seed=0, dtype=BF):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=gen).to(dtype).cuda()
    wgu, wd = ((torch.randn(E, *s, generator=gen) * 0.05).to(dtype).cuda() for s in ((2 * I, H), (H, I)))
    wr = (torch.randn(E, H, generator=gen) * 0.1).to(dtype).cuda()
    return x, wgu, wd, wr


@pytest.mark.parametrize("T,H,I,E,k,align", [(1, 256, 128, 8, 2, 1), (40, 128, 192, 4, 2, 16), (700, 256, 384, 8, 2, 64)])
def test_an_moe_layer_from_its_parts(T, H, I, E, k, align):
    """Router, sort, products, activation and combine, forward and backward,
    against moe_forward and moe_backward's own kernels."""
    x, wgu, wd, wr = layer(T, H, I, E, k, align)
    idx, w, aux, counts = mm.moe_route(x, wr, k, 0.0)
    xs, plan = mm.moe_permute(x, idx, E, align=align)
    gu = mm.grouped_matmul(xs, wgu, plan)
    h = mm.swiglu_act(gu, rows=plan["offsets"][-1:])
    ys = mm.grouped_matmul(h, wd, plan)
    y = mm.moe_unpermute(ys, plan, w)
    Wg, Wu, Wd = [m[:I].contiguous() for m in wgu], [m[I:].contiguous() for m in wgu], list(wd)
    stats = {}
    want, idx2, w2, _ = mm.moe_forward(x, wr, Wg, Wu, Wd, k, coef=0.0, stats=stats)
    same = (idx == idx2).all(1)
    assert same.float().mean() > 0.9
    rms = want.float().square().mean().sqrt()
    # bf16 roundings of gu (twice), h and ys on values about their rms: a few half steps of 2^-8
    assert ((y.float() - want.float())[same].abs().max() / rms) < 16 * 2 ** -8
    dy = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    dys, dw_alpha = mm.moe_unpermute_backward(dy, ys, plan, w)
    dh, dwd = mm.grouped_matmul_backward(dys, h, wd, plan)
    rows = int(plan["offsets"][-1])
    g, u = gu[:rows].float().split(I, 1)
    sig = torch.sigmoid(g)
    dgu = torch.zeros_like(gu)
    dgu[:rows] = torch.cat([dh[:rows].float() * u * sig * (1 + g * (1 - sig)), dh[:rows].float() * g * sig], 1).to(BF)
    dxs, dwgu = mm.grouped_matmul_backward(dgu, xs, wgu, plan)
    if bool(same.all()):
        grads = mm.moe_backward(x, wr, Wg, Wu, Wd, k, 0.0, idx2, w2, stats["probs"], dy, d_aux=0.0)
        for e in range(E):
            for got, ref_ in ((dwd[e], grads["dWd"][e]), (dwgu[e, :I], grads["dWg"][e]), (dwgu[e, I:], grads["dWu"][e])):
                # bf16 roundings of gu, h, dys, dh and dgu on either side: sixteen half steps
                scale = ref_.abs() + ref_.square().mean().sqrt() + 1e-6
                assert ((got - ref_).abs() / scale).max() < 16 * 2 ** -8


def graph_of(call):
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


@pytest.mark.parametrize("T,K,N", [(8, 128, 256), (8, 65, 50), (600, 256, 384), (600, 129, 77)])
def test_captured_and_replayed_with_another_routing(T, K, N):
    """The groups are read on the device, so a replayed graph follows new tables."""
    E, gen = 4, torch.Generator().manual_seed(T)
    w = torch.randn(E, N, K, generator=gen).to(BF).cuda()
    x, dy = torch.randn(T, K, generator=gen).to(BF).cuda(), torch.randn(T, N, generator=gen).to(BF).cuda()
    wq = mm.mx4_quantize(w)
    plan = on_gpu(ref.tables(groups(E, T, "even")))

    def call():
        q = mm.mx4_quantize(x)
        return (mm.grouped_matmul(x, w, plan), *mm.grouped_matmul_backward(dy, x, w, plan), mm.mx4_matmul(x, wq, plan), mm.mx4_matmul(q, wq, plan))

    graph, outs = graph_of(call)
    for how in ("skewed", "one", "even"):
        new = ref.tables(groups(E, T, how, seed=3))
        for key in plan:
            plan[key].copy_(new[key])
        x.copy_(torch.randn(T, K, generator=gen).to(BF))
        graph.replay()
        for got, want in zip(outs, call()):
            assert torch.equal(got, want)


@pytest.mark.parametrize("E,K,N,counts", [(3, 65, 50, [30, 0, 40]), (1, 2050, 72, [700]), (2, 130, 257, [600, 900])])
def test_two_graphs_share_a_workspace(E, K, N, counts):
    """One scratch, with anything in it, and one status word for two captured
    graphs on one stream; the second set holds values that fp32 products on the
    tensor cores turn over to the CUDA cores."""
    gen = torch.Generator().manual_seed(0)
    T = sum(counts)
    plan, status = on_gpu(ref.tables(counts)), mm.new_workspace(256)
    need = [f(T, K, N, E, d) for f in (mm.grouped_matmul_workspace_bytes, mm.grouped_matmul_backward_workspace_bytes) for d in (BF, F32)]
    ws = torch.full((max(*need, mm.mx4_matmul_workspace_bytes(T, K, N, E, False), 256),), 255, dtype=torch.uint8, device="cuda")
    sets = [[torch.randn(*s, generator=gen).cuda() for s in ((T, K), (E, N, K), (T, N))] for _ in range(2)]
    sets[1][0][3, 5] = 2.0 ** -126
    kw = dict(workspace=ws, status_workspace=status)

    def call(*tensors):
        out = []
        for dtype in (BF, F32):
            x, w, dy = (t.to(dtype) for t in tensors)
            out += [mm.grouped_matmul(x, w, plan, **kw), *mm.grouped_matmul_backward(dy, x, w, plan, **kw)]
        x, wq = tensors[0].to(BF), mm.mx4_quantize(tensors[1].to(BF))
        return (*out, mm.mx4_matmul(mm.mx4_quantize(x), wq, plan, **kw), mm.mx4_matmul(x, wq, plan, **kw))

    want = [[t.clone() for t in call(*s)] for s in sets]
    made = [graph_of(lambda s=s: call(*s)) for s in sets]
    for _ in range(3):
        for graph, _ in made:
            graph.replay()
    assert mm.check_status(status) == 0
    for (_, outs), w in zip(made, want):
        for got, ref_ in zip(outs, w):
            assert torch.equal(got, ref_)


def test_another_stream():
    gen = torch.Generator().manual_seed(9)
    x, w, dy = (torch.randn(*s, generator=gen).to(BF).cuda() for s in ((300, 65), (2, 50, 65), (300, 50)))
    plan = on_gpu(ref.tables([100, 200]))

    def call(**kw):
        q, wq = mm.mx4_quantize(x, **kw), mm.mx4_quantize(w, **kw)
        return (mm.grouped_matmul(x, w, plan, **kw), *mm.grouped_matmul_backward(dy, x, w, plan, **kw),
                mm.mx4_matmul(q, wq, plan, **kw), mm.mx4_dequantize(q, **kw))

    want = call()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got = call(stream=stream)
    stream.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_the_same_bits_every_time():
    E, K, N = 8, 512, 768
    gen = torch.Generator().manual_seed(4)
    x, w, dy = (torch.randn(*s, generator=gen).to(BF).cuda() for s in ((900, K), (E, N, K), (900, N)))
    plan = on_gpu(ref.tables(groups(E, 900, "skewed")))
    q, wq = mm.mx4_quantize(x), mm.mx4_quantize(w)
    first = None
    for _ in range(4):
        outs = (mm.grouped_matmul(x, w, plan), *mm.grouped_matmul_backward(dy, x, w, plan), mm.mx4_matmul(q, wq, plan), mm.mx4_matmul(x[:40], wq, on_gpu(ref.tables([5] * 8))),
                mm.mx4_matmul(x, wq, plan), mm.grouped_matmul(x.float(), w.float(), plan), *mm.grouped_matmul_backward(dy[:, :64].float().contiguous(), x.float(), w[0, :64].float()))
        first = first or outs
        for a, b in zip(outs, first):
            assert torch.equal(a, b)


def test_more_elements_than_32_bits_count():
    """Rows behind element 2^31 of every tensor with rows."""
    R, K, N, E = 280_001, 8192, 8192, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(R, K, dtype=BF, device="cuda").normal_(generator=gen)
    w = torch.randn(E, N, K, generator=gen, device="cuda", dtype=F32).mul_(0.02).to(BF)
    # only the last rows belong to a group, so the work stays small
    plan = {"offsets": torch.tensor([R - 300, R - 260, R - 1], dtype=torch.int32, device="cuda"), "counts": torch.tensor([40, 259], dtype=torch.int32, device="cuda")}
    y = torch.full((R, N), 7.0, dtype=BF, device="cuda")
    mm.grouped_matmul(x, w, plan, out=y)
    small = {"offsets": plan["offsets"] - (R - 300), "counts": plan["counts"]}
    want = mm.grouped_matmul(x[R - 300:].clone(), w, small, out=torch.full((300, N), 7.0, dtype=BF, device="cuda"))
    assert torch.equal(y[R - 300:], want) and bool((y[:R - 300] == 7).all())
    dx, dw = mm.grouped_matmul_backward(y, x, w, plan, out=torch.full((R, K), 7.0, dtype=BF, device="cuda"))
    wdx, wdw = mm.grouped_matmul_backward(want, x[R - 300:].clone(), w, small, out=torch.full((300, K), 7.0, dtype=BF, device="cuda"))
    assert torch.equal(dx[R - 300:], wdx) and torch.equal(dw, wdw) and bool((dx[:R - 300] == 7).all())
    del dx, dw
    q, wq = mm.mx4_quantize(x), mm.mx4_quantize(w)
    tail = {"codes": q["codes"][R - 300:].clone(), "exps": q["exps"][:, R - 300:].clone(), "cols": K}
    again = mm.mx4_quantize(x[R - 300:].clone())
    assert torch.equal(tail["codes"], again["codes"]) and torch.equal(tail["exps"], again["exps"])
    back = mm.mx4_dequantize(q)
    assert torch.equal(back[R - 300:], mm.mx4_dequantize(again))
    del back
    mm.mx4_matmul(q, wq, plan, out=y)
    want = mm.mx4_matmul(again, wq, small, out=torch.full((300, N), 7.0, dtype=BF, device="cuda"))
    assert torch.equal(y[R - 300:], want)
    mm.mx4_matmul(x, wq, plan, out=y)
    want = mm.mx4_matmul(x[R - 300:].clone(), wq, small, out=torch.full((300, N), 7.0, dtype=BF, device="cuda"))
    assert torch.equal(y[R - 300:], want)
