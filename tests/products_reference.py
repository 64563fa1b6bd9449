"""Plain 64-bit forms (torch on the CPU) of the experts' products and of
microscaled 4-bit floating point, and the bounds that their tests use.

Bounds.  A result rounded to its type is off by at most half a step of its
value, block_reference.U relative.  A sum of n products in fp32 is off by at
most n + 1 roundings of 2^-24 on the sum of the terms' magnitudes; inside the
tensor cores an addition may cut off instead of rounding, a whole step of
2^-23, so 2 (n + 1) there.  Products of two bf16 or two 4-bit values are
exact in fp32.  fp32 operands of many rows are multiplied there as three bf16
parts each (8 + 8 + 8 bits: all of fp32's 24), without the products of parts
below 2^-25 of the whole: less than one more rounding per product, where the
six products that are added take no more steps than n sums (16 at a time).
"""
import torch

from block_reference import GROUP, U, U32, close, f64

E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def tables(counts, align=1, start=0):
    """offsets and counts of groups of these sizes, each from a multiple of align behind `start`."""
    offsets = [start]
    for n in counts:
        offsets.append(offsets[-1] + -(-n // align) * align)
    return {"offsets": torch.tensor(offsets, dtype=torch.int32), "counts": torch.tensor(counts, dtype=torch.int32)}


def spans(plan, rows):
    """(expert, first row, row behind the last assignment, row behind the group) of every group."""
    if plan is None:
        return [(0, 0, rows, rows)]
    off, cnt = plan["offsets"].tolist(), plan["counts"].tolist()
    return [(e, off[e], off[e] + cnt[e], off[e + 1]) for e in range(len(cnt))]


def matmul(x, w, plan, before):
    """(ys, magnitudes of the terms) from `before`: padding rows zero, rows outside the groups as there."""
    x, w, y = f64(x), f64(w), f64(before).clone()
    w = w if w.dim() == 3 else w[None]
    terms = torch.zeros_like(y)
    for e, a, b, end in spans(plan, x.shape[0]):
        y[a:end] = 0
        y[a:b] = x[a:b] @ w[e].T
        terms[a:b] = x[a:b].abs() @ w[e].T.abs()
    return y, terms


def matmul_backward(dy, x, w, plan, before):
    """((dxs, magnitudes), (dw, magnitudes))."""
    wt = f64(w).transpose(-1, -2)
    dx = matmul(dy, wt, plan, before)
    dy, x = f64(dy), f64(x)
    shape = w.shape if w.dim() == 3 else (1, *w.shape)
    dw, terms = torch.zeros(shape, dtype=torch.float64), torch.zeros(shape, dtype=torch.float64)
    for e, a, b, _ in spans(plan, x.shape[0]):
        dw[e] = dy[a:b].T @ x[a:b]
        terms[e] = dy[a:b].abs().T @ x[a:b].abs()
    return dx, (dw.view(w.shape), terms.view(w.shape))


def close_sum(got, want, terms, n, dtype, what):
    """got within half a step of want and the roundings of a sum of n products."""
    u = U[dtype]
    sums = 2 * (n + 1) * U32 * terms
    close(got, want, u * want.abs() + (1 + u) * sums, what)


# --------------------------------------------- microscaled 4-bit floating point
def nearest_e2m1(v):
    """Codes (without sign) of the nearest e2m1 values of |v| <= 6, ties to the even code."""
    a = v.abs()
    code = torch.zeros(a.shape, dtype=torch.int64)
    for c in range(1, 8):
        middle = (E2M1[c] + E2M1[c - 1]) / 2
        code += ((a > middle) | ((a == middle) & (c % 2 == 0))).long()
    return code


def quantise(x):
    """(codes, exps, values) of x [R, C] from the definition."""
    x = f64(x)
    R, C = x.shape
    G = -(-C // GROUP)
    words = -(-G // 4)
    code = torch.zeros(R, G * GROUP, dtype=torch.int64)
    exps = torch.full((words, R, 4), 127, dtype=torch.uint8)
    values = torch.empty(R, C, dtype=torch.float64)
    for g in range(G):
        v = x[:, g * GROUP:(g + 1) * GROUP]
        bad = ~v.isfinite().all(1)
        amax = torch.where(bad, 0.0, v.abs().amax(1))
        m, p = torch.frexp(amax)                       # 6 2^e = 0.75 2^(e + 3)
        e = torch.where(amax == 0, -126, p.int() - 3 + (m > 0.75).int()).clamp(min=-126)
        scale = torch.ldexp(torch.ones(R, dtype=torch.float64), e)[:, None]
        q = torch.where(bad[:, None], 0.0, v) / scale
        c = nearest_e2m1(q)
        code[:, g * GROUP:g * GROUP + v.shape[1]] = torch.where(bad[:, None], 0, c + 8 * q.signbit().long())
        values[:, g * GROUP:(g + 1) * GROUP] = torch.where(bad[:, None], torch.nan, E2M1[c] * torch.where(q.signbit(), -scale, scale))
        exps[g // 4, :, g % 4] = torch.where(bad, 255, e + 127).to(torch.uint8)
    codes = (code[:, ::2] + 16 * code[:, 1::2]).to(torch.uint8)
    return codes, exps, values


def stored(x):
    """A 4-bit dict of x [..., C] and its values in 64 bits."""
    codes, exps, values = quantise(x.reshape(-1, x.shape[-1]))
    return {"codes": codes.view(*x.shape[:-1], -1), "exps": exps, "cols": x.shape[-1]}, values.view(x.shape)
