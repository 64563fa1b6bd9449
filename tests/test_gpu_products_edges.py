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
    """A result whose products overflow to both sides is not finite, the others are as ever."""
    gen = torch.Generator().manual_seed(rows)
    K, N = 264, 72
    x, w = torch.randn(rows, K, generator=gen), torch.randn(N, K, generator=gen)
    x[3] *= 2.0 ** 100
    w[7] *= 2.0 ** 80
    y = mm.grouped_matmul(x.cuda(), w.cuda()).cpu()
    # products of 2^180 of both signs: their sum, rounded once, is an infinity; added one by one in
    # fp32 they are inf - inf, a NaN.  A finite number is neither.
    assert not bool(y[3, 7].isfinite())
    keep = torch.ones(rows, N, dtype=torch.bool)
    keep[3, 7] = False
    want, terms = ref.matmul(x, w, None, torch.zeros(rows, N))
    ref.close_sum(torch.where(keep, y, 0.0), torch.where(keep, want, 0.0), torch.where(keep, terms, 0.0), K, F32, "ys")


@pytest.mark.parametrize("rows,K,N", [(8, 96, 72), (300, 264, 72), (300, 515, 130), (300, 4096, 130)])
def test_tiny_numbers_do_not_turn_a_call_over(rows, K, N):
    """Tails of a softmax, down to fp32's smallest: the call stays where it is made, which the bits of the other results tell."""
    gen = torch.Generator().manual_seed(rows + N)
    x, w, dy = torch.randn(rows, K, generator=gen), torch.randn(N, K, generator=gen), torch.randn(rows, N, generator=gen)

    def call(x, dy):
        return [t.cpu() for t in (mm.grouped_matmul(x.cuda(), w.cuda()), *mm.grouped_matmul_backward(dy.cuda(), x.cuda(), w.cuda()))]

    clean = call(x, dy)
    small = torch.tensor([2.0 ** -149, -1.3e-33, 2.0 ** -126, 1e-38, -3e-42, 7e-31])
    x[3, :6], dy[3, :6] = small, small
    y, dx, dw = call(x, dy)
    rest = torch.arange(rows) != 3
    assert torch.equal(y[rest], clean[0][rest]) and torch.equal(dx[rest], clean[1][rest]) and torch.equal(dw[6:, 6:], clean[2][6:, 6:])
    for got, (want, terms), n in ((y, ref.matmul(x, w, None, torch.zeros(rows, N)), K), *zip((dx, dw), ref.matmul_backward(dy, x, w, None, torch.zeros(rows, K)), (N, rows))):
        ref.close_sum(got, want, terms, n, F32, "")


@pytest.mark.parametrize("rows,K,N", [(20, 264, 72), (5, 97, 40), (300, 264, 200), (300, 65, 33), (300, 4096, 130)])
@pytest.mark.parametrize("scale", [0, 30, -30])
def test_fp32_products_of_numbers_of_every_size(rows, K, N, scale):
    """24 bits at every exponent from fp32's smallest number to 2^79, times a
    power of two in its place: one term a sum, rounded once where it is subnormal.

    The tensor cores' sums are scaled by 2^48, in which the term is exact."""
    gen = torch.Generator().manual_seed(rows + K + scale)
    x = numbers((2 ** 23, 2 ** 24), gen, rows, K) * torch.exp2(torch.randint(-149, 56 - max(scale, 0), (rows, K), generator=gen).double()).float()
    dy = numbers((2 ** 23, 2 ** 24), gen, rows, N) * torch.exp2(torch.randint(-149, 56 - max(scale, 0), (rows, N), generator=gen).double()).float()
    one = lambda axis, *s: one_each(torch.full(s, 2.0 ** scale), axis, [(0, s[0])], gen)  # noqa: E731
    w, v = one(1, N, K), one(0, N, K)
    y = mm.grouped_matmul(x.cuda(), w.cuda()).cpu()
    dx = mm.grouped_matmul_backward(dy.cuda(), None, v.cuda())[0].cpu()
    assert torch.equal(y, (x.double() @ w.double().T).float()) and torch.equal(dx, (dy.double() @ v.double()).float())
    u = one(0, rows, N)
    dw = mm.grouped_matmul_backward(u.cuda(), x.cuda(), None)[1].cpu()
    assert torch.equal(dw, (u.double().T @ x.double()).float())


# ------------------------------------------------------------ a shared workspace
def calls_with_scratch(gen):
    """Calls that use a workspace, by name: (call with keyword arguments, bytes)."""
    E, K, N, T = 3, 65, 50, 400
    plan = on_gpu(ref.tables([150, 0, 250]))
    x, w, dy = (torch.randn(*s, generator=gen).cuda() for s in ((T, K), (E, N, K), (T, N)))
    xb, wb, dyb = x.to(BF), w.to(BF), dy.to(BF)
    wq, xl, wl = mm.mx4_quantize(wb), torch.randn(300, 4096, generator=gen).to(BF).cuda(), torch.randn(130, 4096, generator=gen).to(BF).cuda()
    wlq = mm.mx4_quantize(wl)
    fw, bw, mx = mm.grouped_matmul_workspace_bytes, mm.grouped_matmul_backward_workspace_bytes, mm.mx4_matmul_workspace_bytes
    return {
        "bf16": (lambda **kw: mm.grouped_matmul(xb, wb, plan, **kw), fw(T, K, N, E, BF)),
        "fp32": (lambda **kw: mm.grouped_matmul(x, w, plan, **kw), fw(T, K, N, E, F32)),
        "parts": (lambda **kw: mm.grouped_matmul(xl, wl, **kw), fw(300, 4096, 130, 1, BF)),
        "bf16 backward": (lambda **kw: mm.grouped_matmul_backward(dyb, xb, wb, plan, **kw), bw(T, K, N, E, BF)),
        "fp32 backward": (lambda **kw: mm.grouped_matmul_backward(dy, x, w, plan, **kw), bw(T, K, N, E, F32)),
        "4-bit weights, converted": (lambda **kw: mm.mx4_matmul(xb, wq, plan, **kw), mx(T, K, N, E, False)),
        "4-bit weights, copied": (lambda **kw: mm.mx4_matmul(xl, wlq, **kw), mx(300, 4096, 130, 1, False)),
    }


def tensors(out):
    return [out] if isinstance(out, torch.Tensor) else [t for t in out if t is not None]


def test_the_header_of_a_workspace_stays_as_it_is():
    """Its 256 bytes hold other calls' state; anything may stand behind them."""
    for name, (call, need) in calls_with_scratch(torch.Generator().manual_seed(21)).items():
        assert need > 256, name
        want = [t.clone() for t in tensors(call())]
        for fill in (0, 255):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            ws[:256] = torch.arange(256, dtype=torch.uint8, device="cuda")
            got = tensors(call(workspace=ws))
            assert torch.equal(ws[:256].cpu(), torch.arange(256, dtype=torch.uint8)), name
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name


def test_one_workspace_for_a_model_and_its_products():
    """The decode kernel of moe_forward keeps the counter of its grid barrier in the header."""
    gen = torch.Generator().manual_seed(22)
    T, H, I, E, k = 16, 256, 128, 4, 2
    x, wr = torch.randn(T, H, generator=gen).to(BF).cuda(), (torch.randn(E, H, generator=gen) * 0.1).to(BF).cuda()
    mats = lambda *s: [(torch.randn(*s, generator=gen) * 0.05).to(BF).cuda() for _ in range(E)]  # noqa: E731
    Wg, Wu, Wd = mats(I, H), mats(I, H), mats(H, I)
    calls = calls_with_scratch(gen)
    want = mm.moe_forward(x, wr, Wg, Wu, Wd, k, coef=0.0)[0]
    ws = mm.new_workspace(max(mm.moe_workspace_bytes(T, H, I, E, k, BF), *(need for _, need in calls.values())))
    for name, (call, _) in calls.items():
        call(workspace=ws)
        assert mm.check_status(ws) == 0, name
        y = mm.moe_forward(x, wr, Wg, Wu, Wd, k, coef=0.0, workspace=ws)[0]
        assert mm.check_status(ws) == 0 and torch.equal(y, want), name


# ------------------------------------------------------------- how exact fp32 is
def off(got, want):
    """Root mean square of the error, relative to the result's."""
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("signs", [True, False])
@pytest.mark.parametrize("rows,K", [(32, 2048), (5, 2049), (400, 96), (400, 768), (400, 4096), (4096, 2048), (4096, 8192)])
def test_fp32_results_are_as_exact_as_fp32(rows, K, signs):
    """Sums of K products, streamed, in tiles and in parts, in every direction.

    An accumulator of the tensor cores takes at most 16 additions (256 summed
    columns), each of which cuts off half a step of 2^-23 on the mean, on a
    partial sum that is half the chunk's on the mean where all terms have one
    sign: 4 * 2^-23 of the chunk, which is the largest of the cases.  Adding the
    chunks rounds K / 256 + 1 times, each time off by 2^-25 in the root mean
    square at most, independent of one another."""
    bound = 4 * 2.0 ** -23 + (K / 256 + 1) ** 0.5 * 2.0 ** -25
    gen = torch.Generator(device="cuda").manual_seed(rows + K)
    make = torch.randn if signs else torch.rand
    a, b, c = (make(*s, generator=gen, device="cuda") for s in ((rows, K), (256, K), (K, 256)))
    assert off(mm.grouped_matmul(a, b), a.double() @ b.double().T) <= bound
    assert off(mm.grouped_matmul_backward(a, None, c)[0], a.double() @ c.double()) <= bound
    d, e = make(K, 320, generator=gen, device="cuda"), c
    for dtype in (F32, BF):
        d, e = d.to(dtype), e.to(dtype)
        assert off(mm.grouped_matmul_backward(d, e, None)[1], d.double().T @ e.double()) <= bound


# Products of one term a sum are exact, whatever the parts that the term is made
# of: each of the six products of parts that are made shows in the result's bits.
KINDS = {
    # the dense factor's values, the others': all three parts times one, one times all three, two times two
    "24 x 1": ((2 ** 23, 2 ** 24), None), "1 x 24": (None, (2 ** 23, 2 ** 24)), "12 x 12": ((2 ** 11, 2 ** 12), (2 ** 11, 2 ** 12))}


def numbers(between, gen, *shape):
    """Odd whole numbers of so many bits, or powers of two, of either sign."""
    sign = 1 - 2 * torch.randint(0, 2, shape, generator=gen)
    if between is None:
        return (sign * torch.exp2(torch.randint(-8, 9, shape, generator=gen).float())).float()
    return (sign * (torch.randint(*between, shape, generator=gen) | 1)).float()


def one_each(m, axis, spans, gen):
    """m with one value along `axis` kept in each of the spans, zeros elsewhere (the spans split the rows)."""
    out = torch.zeros_like(m)
    for a, b in spans:
        if b > a:
            part, n = m[a:b], m[a:b].shape[axis]
            at = torch.randint(0, n, (part.shape[1 - axis],), generator=gen).unsqueeze(axis)
            out[a:b].scatter_(axis, at, part.gather(axis, at))
    return out


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts,K,N", [
    (None, 264, 200), ([9, 0, 17], 2432, 72), (None, 97, 40),                      # few rows
    ([300, 0, 257], 768, 264), ([300, 0, 257], 515, 130), ([70, 3, 200], 65, 33),  # tiles, also with copies of rows
    ([40, 600], 96, 2050), ([300], 4096, 130), ([3000], 72, 60)])                  # sums in parts
def test_fp32_products_use_every_part(counts, K, N, kind):
    left, right = KINDS[kind]
    gen = torch.Generator().manual_seed(K + N)
    plan = None if counts is None else ref.tables(counts, 4)
    R, E = (20, 1) if plan is None else (int(plan["offsets"][-1]), len(counts))
    gplan = on_gpu(plan)
    rows = [(a, b) for _, a, b, _ in ref.spans(plan, R)]

    def weights(between, axis=None):
        w = numbers(between, gen, E * N, K)
        if axis is not None:
            w = one_each(w, axis, [(e * N, (e + 1) * N) for e in range(E)], gen)
        return w.view(E, N, K) if plan is not None else w

    def same(got, want):
        assert torch.equal(got.cpu().double(), want)

    zeros = lambda width: torch.zeros(R, width)  # noqa: E731
    for dense_first in (True, False):            # which factor is dense
        lo, hi = (left, right) if dense_first else (right, left)
        x, dy = numbers(lo, gen, R, K), numbers(lo, gen, R, N)
        w, v = (weights(hi, 1), weights(hi, 0)) if dense_first else (weights(hi), weights(hi))
        if not dense_first:
            x, dy = one_each(x, 1, [(0, R)], gen), one_each(dy, 1, [(0, R)], gen)
        same(mm.grouped_matmul(x.cuda(), w.cuda(), gplan), ref.matmul(x, w, plan, zeros(N))[0])
        same(mm.grouped_matmul_backward(dy.cuda(), None, v.cuda(), gplan)[0], ref.matmul(dy, v.transpose(-1, -2), plan, zeros(K))[0])
        x, dy = numbers(lo, gen, R, K), numbers(hi, gen, R, N)
        if dense_first:
            dy = one_each(dy, 0, rows, gen)      # one row of dy and all of x, or the other way round
        else:
            x = one_each(x, 0, rows, gen)
        same(mm.grouped_matmul_backward(dy.cuda(), x.cuda(), None, gplan)[1], ref.matmul_backward(dy, x, torch.zeros_like(v), plan, zeros(K))[1][0])


def test_two_streams_at_once():
    """Calls that run at the same time, each with a workspace of its own."""
    gen = torch.Generator().manual_seed(33)
    made = [calls_with_scratch(gen) for _ in range(2)]
    want = [{name: [t.clone() for t in tensors(call())] for name, (call, _) in calls.items()} for calls in made]
    spaces = [mm.new_workspace(max(need for _, need in calls.values())) for calls in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = [{}, {}]
    for _ in range(5):
        for name in made[0]:
            for i, (calls, ws, stream) in enumerate(zip(made, spaces, streams)):
                got[i][name] = tensors(calls[name][0](workspace=ws, stream=stream))
    torch.cuda.synchronize()
    for i in range(2):
        assert mm.check_status(spaces[i]) == 0
        for name, outs in want[i].items():
            assert all(torch.equal(a, b) for a, b in zip(got[i][name], outs)), name
