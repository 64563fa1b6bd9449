"""What surrounds the experts' products of an MoE block, with gradients:
block norms with gate and residual scale, tokens sorted by expert and back,
and activations kept in 8 bits.  Argument checks and marshalling only; the
formulas and limits stand in include/mm.h.

Every tensor is contiguous, 16-byte aligned and on the current CUDA device.
Work is enqueued on `stream` (default: the current one); results and scratch
that a call allocates belong to that stream, and inputs made on another stream
must be ordered before the call by the caller.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib as L
from .api import _DTYPES

_GROUP = L.MM_CHECKPOINT_GROUP


def _begin(x, name: str, ndim: int, stream):
    """Checks the leading tensor; returns (dtype code, device, raw stream)."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(x.shape)}")
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {x.dtype}")
    dev = x.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    if stream is not None:
        return dt, dev, stream.cuda_stream
    return dt, dev, torch._C._cuda_getCurrentRawStream(dev)     # current_stream() builds an object: 3 us a call


def _arg(t, name: str, dev: int, dtype, shape):
    """Address of a tensor of exactly this dtype, shape and device (None: null)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor on cuda:{dev}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _empty(shape, dtype, dev, stream):
    """A tensor of the call's own, from the pool of the stream that uses it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _scratch(workspace, need: int, dev: int, stream, name: str):
    """(address, bytes, owner) of the caller's workspace, or of a fresh one where one is needed."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _empty(need, torch.uint8, dev, stream)
        return workspace.data_ptr(), need, workspace
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev:
        raise ValueError(f"workspace of {name} must be a tensor on cuda:{dev}")
    if not workspace.is_contiguous():
        raise ValueError(f"workspace of {name} must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


# ------------------------------------------------------------- block norms
def _norm_parts(dev, dtype, T, H, post_weight, gate, pre_weight):
    """Addresses of the two norm weights and the gate, and whether the gate is per token."""
    per_token = isinstance(gate, torch.Tensor) and gate.dim() == 2
    return (_arg(post_weight, "post_weight", dev, dtype, (H,)),
            _arg(gate, "gate", dev, dtype, (T, H) if per_token else (H,)),
            _arg(pre_weight, "pre_weight", dev, dtype, (H,)), per_token)


def _stat(stats: dict, key: str, T: int, dev: int, stream):
    t = stats.get(key)
    if t is None:
        t = stats[key] = _empty(T, torch.float32, dev, stream)
    return _arg(t, key, dev, torch.float32, (T,))


def block_norm(x: torch.Tensor, f: Optional[torch.Tensor] = None, *,
               post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
               pre_weight: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
               eps: float = 1e-5, out: Optional[torch.Tensor] = None,
               normed: Optional[torch.Tensor] = None, stats: Optional[dict] = None, stream=None):
    """r = residual_scale * x + gate * RMSNorm(f; post_weight) and
    n = RMSNorm(r; pre_weight) in one pass (mm_block_norm): the norm after a
    block with its gate and residual, and the norm before the next one.

    x, f [T, H]; post_weight, pre_weight [H]; gate [H] or [T, H].  Each of the
    three may be None (left out); f None is a plain norm (r is x).  Returns
    (r, n), n None without pre_weight.  out / normed: r and n; `out` may be x
    and `normed` may be f (in place).  With a dict `stats`, it receives
    rstd_post / rstd_pre [T] fp32, which block_norm_backward needs; tensors
    that it holds already are written anew, so give each layer a dict of its
    own until its backward has run.
    """
    dt, dev, raw = _begin(x, "x", 2, stream)
    T, H = shape = x.shape
    dtype = x.dtype
    px = _arg(x, "x", dev, dtype, shape)
    pf = _arg(f, "f", dev, dtype, shape)
    post, g, pre, per_token = _norm_parts(dev, dtype, T, H, post_weight, gate, pre_weight)
    if f is None and out is not None and out is not x:
        raise ValueError("out: without f, r is x itself")
    if pre_weight is None and normed is not None:
        raise ValueError("normed needs pre_weight")
    if f is None:
        out, pout = x, None
    else:
        if out is None:
            out = _empty(shape, dtype, dev, stream)
        pout = _arg(out, "out", dev, dtype, shape)
    if pre_weight is not None and normed is None:
        normed = _empty(shape, dtype, dev, stream)
    post_rstd = pre_rstd = None
    if stats is not None:
        if post is not None:
            post_rstd = _stat(stats, "rstd_post", T, dev, stream)
        if pre is not None:
            pre_rstd = _stat(stats, "rstd_pre", T, dev, stream)
    rc = L.load().mm_block_norm(
        px, pf, post, g, per_token, pre, residual_scale, eps, T, H, dt, pout,
        _arg(normed, "normed", dev, dtype, shape), post_rstd, pre_rstd, raw)
    L.check(rc, "mm_block_norm")
    return out, normed


def block_norm_backward_workspace_bytes(T: int, H: int, dtype: torch.dtype) -> int:
    return int(L.load().mm_block_norm_backward_workspace_bytes(T, H, _DTYPES[dtype]))


def block_norm_backward(dn: Optional[torch.Tensor], dr: Optional[torch.Tensor],
                        r: Optional[torch.Tensor], f: Optional[torch.Tensor],
                        stats: Optional[dict], *,
                        post_weight: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None,
                        pre_weight: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradient of block_norm (mm_block_norm_backward) for dn = dL/dn and
    dr = dL/dr (None: zero), from r, f and the forward's stats.  Returns a
    dict of what has a gradient: dx, df, d_post_weight and d_pre_weight
    (fp32 [H]), d_gate (fp32 [H], or x's dtype [T, H]).  f None: the plain
    norm (r is its x).  Without pre_weight there is no n, and dn must be None."""
    if dn is not None and pre_weight is None:
        raise ValueError("dn needs pre_weight: without it there is no n")
    lead, name = (dn, "dn") if pre_weight is not None else (dr, "dr")
    dt, dev, raw = _begin(lead, name, 2, stream)
    T, H = shape = lead.shape
    dtype = lead.dtype
    post, g, pre, per_token = _norm_parts(dev, dtype, T, H, post_weight, gate, pre_weight)
    if f is None and (post is not None or g is not None or residual_scale != 1.0):
        raise ValueError("post_weight, gate and residual_scale need f")
    rstd = [None, None]
    for i, (key, w) in enumerate((("rstd_post", post), ("rstd_pre", pre))):
        if w is not None:
            if stats is None or stats.get(key) is None:
                raise ValueError(f"stats must hold the forward's {key}")
            rstd[i] = _arg(stats[key], key, dev, torch.float32, (T,))
    pdn = pr = None
    if pre is not None:
        pdn, pr = _arg(dn, "dn", dev, dtype, shape), _arg(r, "r", dev, dtype, shape)
    pdr, pf = _arg(dr, "dr", dev, dtype, shape), _arg(f, "f", dev, dtype, shape)
    lib = L.load()
    sums = post is not None or pre is not None or (g is not None and not per_token)
    need = lib.mm_block_norm_backward_workspace_bytes(T, H, dt) if sums else 0
    pws, nbytes, keep = _scratch(workspace, need, dev, stream, "block_norm_backward")
    out = {"dx": _empty(shape, dtype, dev, stream)}
    pdf = pdpost = pdgate = pdpre = None
    if f is not None:
        t = out["df"] = _empty(shape, dtype, dev, stream)
        pdf = t.data_ptr()
    if post is not None:
        t = out["d_post_weight"] = _empty(H, torch.float32, dev, stream)
        pdpost = t.data_ptr()
    if g is not None:
        t = out["d_gate"] = _empty(shape if per_token else H, dtype if per_token else torch.float32, dev, stream)
        pdgate = t.data_ptr()
    if pre is not None:
        t = out["d_pre_weight"] = _empty(H, torch.float32, dev, stream)
        pdpre = t.data_ptr()
    rc = lib.mm_block_norm_backward(
        pdn, pdr, pr, pf, post, g, per_token, pre, rstd[0], rstd[1], residual_scale, T, H, dt,
        out["dx"].data_ptr(), pdf, pdpost, pdgate, pdpre, pws, nbytes, raw)
    del keep                                    # until the work is enqueued
    L.check(rc, "mm_block_norm_backward")
    return out


# ------------------------------------------------- tokens sorted by expert
def moe_permuted_rows(T: int, E: int, k: int, align: int = 1) -> int:
    """Rows that the sorted tensor of any routing can need (-1: outside the limits)."""
    return int(L.load().mm_moe_permuted_rows(T, E, k, align))


def moe_permute_workspace_bytes(T: int, E: int, k: int) -> int:
    return int(L.load().mm_moe_permute_workspace_bytes(T, E, k))


def _table(plan: dict, key: str, shape, dev: int, stream) -> int:
    """Address of an index table of the plan, made where it is not there."""
    t = plan.get(key)
    if t is not None:
        return _arg(t, key, dev, torch.int32, shape)
    t = plan[key] = _empty(shape, torch.int32, dev, stream)
    return t.data_ptr()


def moe_permute(x: torch.Tensor, topk_idx: torch.Tensor, E: int, *, align: int = 1,
                out: Optional[torch.Tensor] = None, plan: Optional[dict] = None,
                workspace: Optional[torch.Tensor] = None, stream=None):
    """Rows of x [T, H] sorted by expert (mm_moe_permute) for topk_idx [T, k]
    int32; an index outside [0, E) drops the assignment.  Returns (xs [R, H],
    plan), R = moe_permuted_rows(T, E, k, align); plan (a dict, whose tensors
    are reused when it is given) holds offsets [E + 1], counts [E], perm [R]
    and pos [T, k], all int32.  Rows from offsets[E] on are left as they were."""
    dt, dev, raw = _begin(x, "x", 2, stream)
    T, H = x.shape
    if not isinstance(topk_idx, torch.Tensor) or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, k]")
    k = topk_idx.shape[1]
    px = _arg(x, "x", dev, x.dtype, (T, H))
    pi = _arg(topk_idx, "topk_idx", dev, torch.int32, (T, k))
    lib = L.load()
    if E < 1 or k < 1 or align < 1:
        raise L.MMError(L.MM_ERR_INVALID_ARG, "mm_moe_permute")
    R = lib.mm_moe_permuted_rows(T, E, k, align)
    if R < 0:
        raise L.MMError(L.MM_ERR_UNSUPPORTED, "mm_moe_permute")
    plan = {} if plan is None else plan
    pws, nbytes, keep = _scratch(workspace, lib.mm_moe_permute_workspace_bytes(T, E, k), dev, stream, "moe_permute")
    if out is None:
        out = _empty((R, H), x.dtype, dev, stream)
    po = _arg(out, "out", dev, x.dtype, (R, H))
    rc = lib.mm_moe_permute(
        px, pi, T, H, E, k, align, dt, po, _table(plan, "offsets", (E + 1,), dev, stream),
        _table(plan, "counts", (E,), dev, stream), _table(plan, "perm", (R,), dev, stream),
        _table(plan, "pos", (T, k), dev, stream), pws, nbytes, raw)
    del keep                                    # until the work is enqueued
    L.check(rc, "mm_moe_permute")
    return out, plan


def _combine(rows, name, plan, topk_w, out, stream):
    dt, dev, raw = _begin(rows, name, 2, stream)
    R, H = rows.shape
    pos = plan["pos"]
    T, k = pos.shape
    pr = _arg(rows, name, dev, rows.dtype, (R, H))
    pp = _arg(pos, "pos", dev, torch.int32, (T, k))
    pw = _arg(topk_w, "topk_w", dev, torch.float32, (T, k))
    if out is None:
        out = _empty((T, H), rows.dtype, dev, stream)
    rc = L.load().mm_moe_unpermute(pr, pp, pw, T, H, k, R, dt,
                                   _arg(out, "out", dev, rows.dtype, (T, H)), raw)
    L.check(rc, "mm_moe_unpermute")
    return out


def moe_unpermute(ys: torch.Tensor, plan: dict, topk_w: torch.Tensor, *,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y[t] = sum_s topk_w[t, s] ys[pos[t, s]] (mm_moe_unpermute); a token with
    every assignment dropped gets zeros."""
    if topk_w is None:
        raise ValueError("topk_w is needed")
    return _combine(ys, "ys", plan, topk_w, out, stream)


def moe_permute_backward(dxs: torch.Tensor, plan: dict, *, out: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """Gradient of moe_permute: dx[t] = sum_s dxs[pos[t, s]]."""
    return _combine(dxs, "dxs", plan, None, out, stream)


def moe_unpermute_backward(dy: torch.Tensor, ys: Optional[torch.Tensor], plan: dict,
                           topk_w: Optional[torch.Tensor], *, out: Optional[torch.Tensor] = None,
                           stream=None):
    """Gradient of moe_unpermute (mm_moe_unpermute_backward): (dys [R, H],
    dw [T, k] fp32).  Rows of dys from offsets[E] on are left as they were
    (give `out`).  topk_w None: dys[pos] = dy and dw None (the permute of dy by
    the plan's order; ys is not read)."""
    dt, dev, raw = _begin(dy, "dy", 2, stream)
    T, H = dy.shape
    pos, counts = plan["pos"], plan["counts"]
    k, E, R = pos.shape[-1], counts.shape[0], plan["perm"].shape[0]
    weighted = topk_w is not None
    if weighted and ys is None:
        raise ValueError("ys is needed with topk_w")
    args = (_arg(dy, "dy", dev, dy.dtype, (T, H)),
            _arg(ys, "ys", dev, dy.dtype, (R, H)) if weighted else None,
            _arg(pos, "pos", dev, torch.int32, (T, k)),
            _arg(topk_w, "topk_w", dev, torch.float32, (T, k)),
            _arg(plan["offsets"], "offsets", dev, torch.int32, (E + 1,)),
            _arg(counts, "counts", dev, torch.int32, (E,)))
    if out is None:
        out = _empty((R, H), dy.dtype, dev, stream)
    dw = _empty((T, k), torch.float32, dev, stream) if weighted else None
    rc = L.load().mm_moe_unpermute_backward(
        *args, T, H, E, k, R, dt, _arg(out, "out", dev, dy.dtype, (R, H)),
        dw.data_ptr() if weighted else None, raw)
    L.check(rc, "mm_moe_unpermute_backward")
    return out, dw


# ----------------------------------------------------- activations in 8 bits
def _groups(cols: int) -> int:
    return -(-cols // _GROUP)


def checkpoint_pack(x: torch.Tensor, *, stream=None) -> dict:
    """x [R, C] kept in 8 bits (mm_checkpoint_pack): a dict of codes [R, C]
    (float8_e4m3fn), exps [R, ceil(C / 32)] (uint8, biased powers of two, one
    per group of 32 columns) and segments 1."""
    dt, dev, raw = _begin(x, "x", 2, stream)
    R, C = x.shape
    px = _arg(x, "x", dev, x.dtype, (R, C))
    codes = _empty((R, C), torch.float8_e4m3fn, dev, stream)
    exps = _empty((R, _groups(C)), torch.uint8, dev, stream)
    rc = L.load().mm_checkpoint_pack(px, R, C, dt, codes.data_ptr(), exps.data_ptr(), raw)
    L.check(rc, "mm_checkpoint_pack")
    return {"codes": codes, "exps": exps, "segments": 1}


def _checkpoint_args(checkpoint: dict):
    """(codes, exps, segments, R, columns of a segment), the shapes checked against each other."""
    codes, exps, seg = checkpoint["codes"], checkpoint["exps"], checkpoint["segments"]
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise ValueError("codes must be [R, C]")
    R, C = codes.shape
    if seg not in (1, 2) or C % seg:
        raise ValueError(f"{C} columns do not make {seg} segments")
    return codes, exps, seg, R, C // seg


def checkpoint_unpack(checkpoint: dict, dtype: torch.dtype = torch.bfloat16, *,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values a checkpoint stands for (mm_checkpoint_unpack), in `dtype`."""
    codes, exps, seg, R, C = _checkpoint_args(checkpoint)
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    if out is None:
        out = _empty((R, seg * C), dtype, codes.device, stream)
    dt, dev, raw = _begin(out, "out", 2, stream)
    rc = L.load().mm_checkpoint_unpack(
        _arg(codes, "codes", dev, torch.float8_e4m3fn, (R, seg * C)),
        _arg(exps, "exps", dev, torch.uint8, (R, seg * _groups(C))), R * seg, C, dt,
        _arg(out, "out", dev, dtype, (R, seg * C)), raw)
    L.check(rc, "mm_checkpoint_unpack")
    return out


def _rows_arg(rows, dev):
    return None if rows is None else _arg(rows, "rows", dev, torch.int32, (1,))


def swiglu_act(gu: torch.Tensor, *, checkpoint: Optional[dict] = None,
               out: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """h = SiLU(g) u [R, I] of gu [R, 2I], g in the first I columns
    (mm_swiglu_act).  With a dict `checkpoint`, g and u are also kept in 8 bits
    in it: codes [R, 2I], exps [R, 2 ceil(I / 32)], segments 2 (tensors already
    there are reused).  rows (int32 [1] on the device, such as a plan's
    offsets[-1:]): rows from that one on are left alone."""
    dt, dev, raw = _begin(gu, "gu", 2, stream)
    R, two_i = gu.shape
    if two_i % 2:
        raise ValueError("gu must have an even number of columns")
    I = two_i // 2
    pg = _arg(gu, "gu", dev, gu.dtype, (R, two_i))
    pr = _rows_arg(rows, dev)
    pc = pe = None
    if out is None:
        out = _empty((R, I), gu.dtype, dev, stream)
    if checkpoint is not None:
        codes, exps = checkpoint.get("codes"), checkpoint.get("exps")
        if codes is None:
            codes = _empty((R, two_i), torch.float8_e4m3fn, dev, stream)
        if exps is None:
            exps = _empty((R, 2 * _groups(I)), torch.uint8, dev, stream)
        pc = _arg(codes, "codes", dev, torch.float8_e4m3fn, (R, two_i))
        pe = _arg(exps, "exps", dev, torch.uint8, (R, 2 * _groups(I)))
    rc = L.load().mm_swiglu_act(pg, R, I, dt, pr, _arg(out, "out", dev, gu.dtype, (R, I)), pc, pe, raw)
    L.check(rc, "mm_swiglu_act")
    if checkpoint is not None:                  # not before: a refused call leaves it as it was
        checkpoint.update(codes=codes, exps=exps, segments=2)
    return out


def swiglu_act_backward(checkpoint: dict, dh: torch.Tensor, *, want_h: bool = True,
                        out: Optional[torch.Tensor] = None, h_out: Optional[torch.Tensor] = None,
                        rows: Optional[torch.Tensor] = None, stream=None):
    """(dgu [R, 2I], h [R, I]) from the 8-bit g and u that swiglu_act kept, for
    dh [R, I] (mm_swiglu_act_backward); h, the operand of the down weights'
    gradient, is left out with want_h=False.  rows as in swiglu_act."""
    codes, exps, seg, R, I = _checkpoint_args(checkpoint)
    if seg != 2:
        raise ValueError("the checkpoint holds no g and u (segments 2)")
    dt, dev, raw = _begin(dh, "dh", 2, stream)
    pd = _arg(dh, "dh", dev, dh.dtype, (R, I))
    if not want_h and h_out is not None:
        raise ValueError("h_out needs want_h")
    if out is None:
        out = _empty((R, 2 * I), dh.dtype, dev, stream)
    if want_h and h_out is None:
        h_out = _empty((R, I), dh.dtype, dev, stream)
    rc = L.load().mm_swiglu_act_backward(
        _arg(codes, "codes", dev, torch.float8_e4m3fn, (R, 2 * I)),
        _arg(exps, "exps", dev, torch.uint8, (R, 2 * _groups(I))), pd, R, I, dt, _rows_arg(rows, dev),
        _arg(out, "out", dev, dh.dtype, (R, 2 * I)), _arg(h_out, "h_out", dev, dh.dtype, (R, I)), raw)
    L.check(rc, "mm_swiglu_act_backward")
    return out, h_out
