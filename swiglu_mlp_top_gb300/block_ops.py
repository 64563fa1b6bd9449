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

import contextlib
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
    dev = x.device
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {dev}, the current device is cuda:{torch.cuda.current_device()}")
    s = stream if stream is not None else torch.cuda.current_stream()
    return dt, dev, s.cuda_stream


def _arg(t, name: str, dev, dtype, shape):
    """Address of a tensor of exactly this dtype, shape and device (None: null)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device != dev:
        raise ValueError(f"{name} must be a tensor on {dev}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _on(stream):
    """Where a call's own tensors are allocated: the pool of the stream that uses them."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _scratch(workspace, need: int, dev, name: str):
    """(tensor, bytes): the caller's workspace, or a fresh one (no header state is needed)."""
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif not isinstance(workspace, torch.Tensor) or workspace.device != dev:
        raise ValueError(f"workspace of {name} must be a tensor on {dev}")
    elif not workspace.is_contiguous():
        raise ValueError(f"workspace of {name} must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


# ------------------------------------------------------------- block norms
def _norm_parts(dev, dtype, T, H, post_weight, gate, pre_weight):
    """Addresses of the two norm weights and the gate, and whether the gate is per token."""
    per_token = isinstance(gate, torch.Tensor) and gate.dim() == 2
    return (_arg(post_weight, "post_weight", dev, dtype, (H,)),
            _arg(gate, "gate", dev, dtype, (T, H) if per_token else (H,)),
            _arg(pre_weight, "pre_weight", dev, dtype, (H,)), per_token)


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
    rstd_post / rstd_pre [T] fp32, which block_norm_backward needs.
    """
    dt, dev, raw = _begin(x, "x", 2, stream)
    T, H = x.shape
    dtype = x.dtype
    px = _arg(x, "x", dev, dtype, (T, H))
    pf = _arg(f, "f", dev, dtype, (T, H))
    post, g, pre, per_token = _norm_parts(dev, dtype, T, H, post_weight, gate, pre_weight)
    if f is None and out is not None and out is not x:
        raise ValueError("out: without f, r is x itself")
    if pre_weight is None and normed is not None:
        raise ValueError("normed needs pre_weight")
    with _on(stream):
        if f is None:
            out = x
        elif out is None:
            out = torch.empty_like(x)
        if pre_weight is not None and normed is None:
            normed = torch.empty_like(x)
        rstd = [None, None]
        if stats is not None:
            for i, (key, w) in enumerate((("rstd_post", post_weight), ("rstd_pre", pre_weight))):
                if w is None:
                    continue
                if stats.get(key) is None:
                    stats[key] = torch.empty(T, dtype=torch.float32, device=dev)
                rstd[i] = _arg(stats[key], key, dev, torch.float32, (T,))
    rc = L.load().mm_block_norm(
        px, pf, post, g, per_token, pre, residual_scale, eps, T, H, dt,
        None if f is None else _arg(out, "out", dev, dtype, (T, H)),
        _arg(normed, "normed", dev, dtype, (T, H)), rstd[0], rstd[1], raw)
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
    norm (r is its x)."""
    lead, name = (dn, "dn") if pre_weight is not None else (dr, "dr")
    dt, dev, raw = _begin(lead, name, 2, stream)
    T, H = lead.shape
    dtype = lead.dtype
    post, g, pre, per_token = _norm_parts(dev, dtype, T, H, post_weight, gate, pre_weight)
    if f is None and (post_weight is not None or gate is not None or residual_scale != 1.0):
        raise ValueError("post_weight, gate and residual_scale need f")
    rstd = [None, None]
    for i, (key, w) in enumerate((("rstd_post", post_weight), ("rstd_pre", pre_weight))):
        if w is not None:
            if stats is None or stats.get(key) is None:
                raise ValueError(f"stats must hold the forward's {key}")
            rstd[i] = _arg(stats[key], key, dev, torch.float32, (T,))
    pdn = _arg(dn, "dn", dev, dtype, (T, H)) if pre_weight is not None else None
    pr = _arg(r, "r", dev, dtype, (T, H)) if pre_weight is not None else None
    pdr = _arg(dr, "dr", dev, dtype, (T, H))
    pf = _arg(f, "f", dev, dtype, (T, H))
    lib = L.load()
    need = lib.mm_block_norm_backward_workspace_bytes(T, H, dt)
    with _on(stream):
        workspace, nbytes = _scratch(workspace, need, dev, "block_norm_backward")
        out = {"dx": torch.empty_like(lead)}
        if f is not None:
            out["df"] = torch.empty_like(lead)
        if post_weight is not None:
            out["d_post_weight"] = torch.empty(H, dtype=torch.float32, device=dev)
        if gate is not None:
            out["d_gate"] = torch.empty((T, H) if per_token else (H,), device=dev,
                                        dtype=dtype if per_token else torch.float32)
        if pre_weight is not None:
            out["d_pre_weight"] = torch.empty(H, dtype=torch.float32, device=dev)

    def at(key):
        return out[key].data_ptr() if key in out else None

    rc = lib.mm_block_norm_backward(
        pdn, pdr, pr, pf, post, g, per_token, pre, rstd[0], rstd[1], residual_scale, T, H, dt,
        at("dx"), at("df"), at("d_post_weight"), at("d_gate"), at("d_pre_weight"),
        workspace.data_ptr(), nbytes, raw)
    L.check(rc, "mm_block_norm_backward")
    return out


# ------------------------------------------------- tokens sorted by expert
def moe_permuted_rows(T: int, E: int, k: int, align: int = 1) -> int:
    """Rows that the sorted tensor of any routing can need (-1: outside the limits)."""
    return int(L.load().mm_moe_permuted_rows(T, E, k, align))


def moe_permute_workspace_bytes(T: int, E: int, k: int) -> int:
    return int(L.load().mm_moe_permute_workspace_bytes(T, E, k))


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
    with _on(stream):
        workspace, nbytes = _scratch(workspace, lib.mm_moe_permute_workspace_bytes(T, E, k), dev,
                                     "moe_permute")
        if out is None:
            out = torch.empty(R, H, dtype=x.dtype, device=dev)
        ptrs = []
        for key, shape in (("offsets", (E + 1,)), ("counts", (E,)), ("perm", (R,)), ("pos", (T, k))):
            if plan.get(key) is None:
                plan[key] = torch.empty(shape, dtype=torch.int32, device=dev)
            ptrs.append(_arg(plan[key], key, dev, torch.int32, shape))
    rc = lib.mm_moe_permute(px, pi, T, H, E, k, align, dt, _arg(out, "out", dev, x.dtype, (R, H)),
                            *ptrs, workspace.data_ptr(), nbytes, raw)
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
        with _on(stream):
            out = torch.empty(T, H, dtype=rows.dtype, device=dev)
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
    with _on(stream):
        if out is None:
            out = torch.empty(R, H, dtype=dy.dtype, device=dev)
        dw = torch.empty(T, k, dtype=torch.float32, device=dev) if weighted else None
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
    with _on(stream):
        codes = torch.empty(R, C, dtype=torch.float8_e4m3fn, device=dev)
        exps = torch.empty(R, _groups(C), dtype=torch.uint8, device=dev)
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
        with _on(stream):
            out = torch.empty(R, seg * C, dtype=dtype, device=codes.device)
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
    with _on(stream):
        if out is None:
            out = torch.empty(R, I, dtype=gu.dtype, device=dev)
        if checkpoint is not None:
            if checkpoint.get("codes") is None:
                checkpoint["codes"] = torch.empty(R, two_i, dtype=torch.float8_e4m3fn, device=dev)
            if checkpoint.get("exps") is None:
                checkpoint["exps"] = torch.empty(R, 2 * _groups(I), dtype=torch.uint8, device=dev)
            checkpoint["segments"] = 2
            pc = _arg(checkpoint["codes"], "codes", dev, torch.float8_e4m3fn, (R, two_i))
            pe = _arg(checkpoint["exps"], "exps", dev, torch.uint8, (R, 2 * _groups(I)))
    rc = L.load().mm_swiglu_act(pg, R, I, dt, pr, _arg(out, "out", dev, gu.dtype, (R, I)), pc, pe, raw)
    L.check(rc, "mm_swiglu_act")
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
    with _on(stream):
        if out is None:
            out = torch.empty(R, 2 * I, dtype=dh.dtype, device=dev)
        if want_h and h_out is None:
            h_out = torch.empty(R, I, dtype=dh.dtype, device=dev)
    rc = L.load().mm_swiglu_act_backward(
        _arg(codes, "codes", dev, torch.float8_e4m3fn, (R, 2 * I)),
        _arg(exps, "exps", dev, torch.uint8, (R, 2 * _groups(I))), pd, R, I, dt, _rows_arg(rows, dev),
        _arg(out, "out", dev, dh.dtype, (R, 2 * I)), _arg(h_out, "h_out", dev, dh.dtype, (R, I)), raw)
    L.check(rc, "mm_swiglu_act_backward")
    return out, h_out
