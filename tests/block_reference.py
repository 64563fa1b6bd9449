"""Plain 64-bit forms (torch on the CPU) of the operators around the experts'
products, and the error bounds that their tests use.

Bounds.  A result rounded to its type is off by at most half a step of its
value, U[dtype] = finfo.eps / 2 relative.  Before that rounding the kernels
compute in fp32: a product or sum of terms with magnitudes that add up to A is
off by at most c * 2^-24 * A, where c counts the roundings on the longest way
from an input to the result (a sum of n terms in any order: n).
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -24
GROUP = 32


def f64(t):
    return None if t is None else t.detach().cpu().double()


def close(got, want, bound, what=""):
    """Every element of got within `bound` (a tensor of the same shape) of want."""
    got, want = f64(got), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if got.numel() == 0:
        return
    over = (got - want).abs() - bound
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    worst = over.max().item()
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} off, the worst by {worst:g} more than allowed"


# -------------------------------------------------------------- block norms
def norm_forward(x, f, post, gate, pre, s, eps, r_stored=None):
    """64-bit r, n, rstd of f and r; n is the norm of r_stored (default: r)."""
    x, f, post, gate, pre = map(f64, (x, f, post, gate, pre))
    out = {}
    r = x
    if f is not None:
        p = f
        if post is not None:
            out["rstd_post"] = 1 / (f.square().mean(1) + eps).sqrt()
            p = f * out["rstd_post"][:, None] * post
        if gate is not None:
            p = p * gate
        r = s * x + p
        out["r_terms"] = abs(s) * x.abs() + p.abs()
    out["r"] = r
    if pre is not None:
        rs = r if r_stored is None else f64(r_stored)
        out["rstd_pre"] = 1 / (rs.square().mean(1) + eps).sqrt()
        out["n"] = rs * out["rstd_pre"][:, None] * pre
    return out


def norm_backward(dn, dr, r, f, post, gate, pre, s, rf, rr):
    """64-bit gradients by the formulas, and for each the magnitudes of its
    terms (key + "_terms") for the bounds."""
    dn, dr, r, f, post, gate, pre, rf, rr = map(f64, (dn, dr, r, f, post, gate, pre, rf, rr))
    out = {}
    shape = (dn if dr is None else dr).shape
    D = torch.zeros(shape, dtype=torch.float64) if dr is None else dr
    A = D.abs()
    if pre is not None:
        v, rr = dn * pre, rr[:, None]
        D = D + rr * v - r * rr ** 3 * (r * v).mean(1, keepdim=True)
        A = A + (rr * v).abs() + r.abs() * rr ** 3 * (r * v).abs().mean(1, keepdim=True)
        out["d_pre_weight"] = (dn * r * rr).sum(0)
        out["d_pre_weight_terms"] = (dn * r * rr).abs().sum(0)
    out["dx"], out["dx_terms"] = s * D, abs(s) * A
    if f is None:
        return out
    unit = f if post is None else f * rf[:, None]
    p = unit if post is None else unit * post
    q, Q = (D, A) if gate is None else (D * gate, A * gate.abs())
    if gate is not None:
        dg, dgt = D * p, A * p.abs()
        out["d_gate"], out["d_gate_terms"] = (dg, dgt) if gate.dim() == 2 else (dg.sum(0), dgt.sum(0))
    if post is not None:
        rf = rf[:, None]
        out["d_post_weight"], out["d_post_weight_terms"] = (q * unit).sum(0), (Q * unit.abs()).sum(0)
        v, V = q * post, Q * post.abs()
        out["df"] = rf * v - f * rf ** 3 * (f * v).mean(1, keepdim=True)
        out["df_terms"] = rf * V + f.abs() * rf ** 3 * (f.abs() * V).mean(1, keepdim=True)
    else:
        out["df"], out["df_terms"] = q, Q
    return out


# ------------------------------------------------- tokens sorted by expert
def sort_plan(idx, E, align, rows):
    """offsets, counts, perm, pos of topk_idx [T, k], assignment by assignment."""
    flat = idx.reshape(-1).tolist()
    groups = [[a for a, e in enumerate(flat) if e == g] for g in range(E)]
    offsets, perm, pos = [0], [-1] * rows, [-1] * len(flat)
    for g in groups:
        for i, a in enumerate(g):
            perm[offsets[-1] + i] = a
            pos[a] = offsets[-1] + i
        offsets.append(offsets[-1] + math.ceil(len(g) / align) * align)
    as_int = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"offsets": as_int(offsets), "counts": as_int([len(g) for g in groups]),
            "perm": as_int(perm), "pos": as_int(pos).view(idx.shape)}


def gathered(rows, pos):
    """[T, k, H] of the rows at pos, zeros where pos is -1."""
    got = f64(rows)[pos.clamp(min=0).long()]
    return got * (pos >= 0)[..., None]


# ----------------------------------------------------- activations in 8 bits
#: e4m3 magnitudes by code, from the format's definition (bias 7, subnormals, 0x7f NaN).
E4M3 = torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) / 8 * 2.0 ** ((c >> 3) - 7)
                     for c in range(127)], dtype=torch.float64)


def nearest_e4m3(v):
    """Nearest e4m3 value, ties to the even code, for |v| <= 448 (NaN stays)."""
    a = v.abs()
    hi = torch.searchsorted(E4M3, a.nan_to_num(0.0).contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.where(v.isnan(), v, E4M3[code] * torch.where(v.signbit(), -1.0, 1.0))


def checkpoint(x):
    """(code values, biased exponents, values) of x [R, C] from the definition."""
    x = f64(x)
    R, C = x.shape
    G = -(-C // GROUP)
    codes, values = torch.empty_like(x), torch.empty_like(x)
    exps = torch.empty(R, G, dtype=torch.uint8)
    for g in range(G):
        v = x[:, g * GROUP:(g + 1) * GROUP]
        amax = torch.where(v.isfinite(), v.abs(), 0.0).amax(1)
        m, p = torch.frexp(amax)
        e = torch.where(amax == 0, -126, p.int() - 9 + (m > 0.875).int()).clamp(min=-126)
        scale = torch.ldexp(torch.ones(R, dtype=torch.float64), e)[:, None]
        q = nearest_e4m3(torch.where(v.isfinite(), v, torch.nan) / scale)
        codes[:, g * GROUP:(g + 1) * GROUP] = q
        values[:, g * GROUP:(g + 1) * GROUP] = q * scale
        exps[:, g] = (e + 127).to(torch.uint8)
    return codes, exps, values


def swiglu(g, u):
    return g * torch.sigmoid(g) * u


def swiglu_backward(g, u, dh):
    """(dG, dU) and the magnitudes of dG's terms."""
    s, c = torch.sigmoid(g), torch.sigmoid(-g)
    return dh * u * s * (1 + g * c), dh * g * s, (dh * u).abs() * s * (1 + g.abs() * c)
