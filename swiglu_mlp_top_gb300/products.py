"""The experts' matrix products on rows sorted by expert, with gradients, in
bf16, fp32 and microscaled 4-bit floating point.  Argument checks and
marshalling only; the formulas and limits stand in include/mm.h.

Tensors, devices and streams as in block_ops.py.  `plan` is what moe_permute
returns (its offsets and counts); without one, all rows take one matrix.
check_status() of `workspace` or, where one is given, of `status_workspace`
(new_workspace(256)) tells of a device wait that gave up; without either
nothing does.  A `workspace` comes from new_workspace() and may be shared with
other calls on its stream.
"""
from __future__ import annotations

from functools import lru_cache
from typing import Optional, Union

import torch

from . import _lib as L
from .api import _DTYPES
from .block_ops import _arg, _begin, _empty, _rows_arg, _scratch

_GROUP = 32          # columns that share a scale
_WORD = 4            # scales of a row next to each other


@lru_cache(maxsize=1024)
def _need(query: str, dev: int, *sizes) -> int:
    """Scratch of a call on the current device `dev`: a function of the sizes alone."""
    return getattr(L.load(), query)(*sizes)


def _device(t, name: str, stream):
    """(device, raw stream) of a call's leading tensor, whatever its type."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev, stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)


def _plan_args(plan: Optional[dict], dev: int):
    """(offsets, counts, E) of a plan; (None, None, 1) without."""
    if plan is None:
        return None, None, 1
    counts = plan["counts"]
    if not isinstance(counts, torch.Tensor) or counts.dim() != 1:
        raise ValueError("counts must be [E]")
    E = counts.shape[0]
    return (_arg(plan["offsets"], "offsets", dev, torch.int32, (E + 1,)),
            _arg(counts, "counts", dev, torch.int32, (E,)), E)


def _weight_shape(E: int, grouped: bool, N: int, K: int):
    return (E, N, K) if grouped else (N, K)


def _weight_rows(shape, plan, name: str) -> int:
    """N of a weight tensor's shape: [E, N, K] with a plan, [N, K] without."""
    if len(shape) != (2 if plan is None else 3):
        raise ValueError(f"{name} must be {'[N, K]' if plan is None else '[E, N, K]'}, got {list(shape)}")
    return shape[-2]


def _status_arg(status, dev: int):
    if status is None:
        return None
    if not isinstance(status, torch.Tensor) or status.get_device() != dev:
        raise ValueError(f"status_workspace must be a tensor on cuda:{dev}")
    if not status.is_contiguous() or status.numel() * status.element_size() < 256:
        raise ValueError("status_workspace must be contiguous and hold 256 bytes")
    return status.data_ptr()


# ------------------------------------------------------ products by expert
def grouped_matmul_workspace_bytes(rows: int, K: int, N: int, E: int, dtype: torch.dtype) -> int:
    return int(L.load().mm_grouped_matmul_workspace_bytes(rows, K, N, E, _DTYPES[dtype]))


def grouped_matmul(xs: torch.Tensor, w: torch.Tensor, plan: Optional[dict] = None, *,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   status_workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """ys [R, N]: each row of xs [R, K] times the matrix of its expert, w
    [E, N, K] in xs's dtype (mm_grouped_matmul); without a plan, w [N, K] for
    all rows.  Padding rows of a group become zeros, rows behind the last group
    are left as they were (give `out`)."""
    dt, dev, raw = _begin(xs, "xs", 2, stream)
    R, K = xs.shape
    off, cnt, E = _plan_args(plan, dev)
    if not isinstance(w, torch.Tensor):
        raise ValueError(f"w must be a tensor on cuda:{dev}")
    N = _weight_rows(w.shape, plan, "w")
    px = _arg(xs, "xs", dev, xs.dtype, (R, K))
    pw = _arg(w, "w", dev, xs.dtype, _weight_shape(E, plan is not None, N, K))
    lib = L.load()
    need = _need("mm_grouped_matmul_workspace_bytes", dev, R, K, N, E, dt)
    ps = _status_arg(status_workspace, dev)
    pws, nbytes, keep = _scratch(workspace, need, dev, stream, "grouped_matmul")
    if out is None:
        out = _empty((R, N), xs.dtype, dev, stream)
    rc = lib.mm_grouped_matmul(px, pw, off, cnt, R, K, N, E, dt, _arg(out, "out", dev, xs.dtype, (R, N)),
                               pws, nbytes, ps, raw)
    del keep                                    # until the work is enqueued
    L.check(rc, "mm_grouped_matmul")
    return out


def grouped_matmul_backward_workspace_bytes(rows: int, K: int, N: int, E: int, dtype: torch.dtype) -> int:
    return int(L.load().mm_grouped_matmul_backward_workspace_bytes(rows, K, N, E, _DTYPES[dtype]))


def grouped_matmul_backward(dys: torch.Tensor, xs: Optional[torch.Tensor], w: Optional[torch.Tensor],
                            plan: Optional[dict] = None, *, out: Optional[torch.Tensor] = None,
                            dw: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                            status_workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of grouped_matmul for dys [R, N] (mm_grouped_matmul_backward):
    (dxs [R, K], dw fp32 [E, N, K], or [N, K] without a plan).  w None: dxs is
    None and only dw is made; xs None: dw is None.  Padding rows of dxs become
    zeros, rows behind the last group are left as they were (give `out`); dw is
    overwritten."""
    dt, dev, raw = _begin(dys, "dys", 2, stream)
    R, N = dys.shape
    off, cnt, E = _plan_args(plan, dev)
    if xs is None and w is None:
        raise ValueError("xs or w is needed")
    for t, name in ((xs, "xs"), (w, "w")):
        if t is not None and not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a tensor on cuda:{dev}")
    if w is not None:
        _weight_rows(w.shape, plan, "w")
    K = (xs if w is None else w).shape[-1]
    shape = _weight_shape(E, plan is not None, N, K)
    pd = _arg(dys, "dys", dev, dys.dtype, (R, N))
    px = _arg(xs, "xs", dev, dys.dtype, (R, K))
    pw = _arg(w, "w", dev, dys.dtype, shape)
    if out is not None and w is None:
        raise ValueError("out needs w")
    if dw is not None and xs is None:
        raise ValueError("dw needs xs")
    lib = L.load()
    need = _need("mm_grouped_matmul_backward_workspace_bytes", dev, R, K, N, E, dt)
    ps = _status_arg(status_workspace, dev)
    pws, nbytes, keep = _scratch(workspace, need, dev, stream, "grouped_matmul_backward")
    if w is not None and out is None:
        out = _empty((R, K), dys.dtype, dev, stream)
    if xs is not None and dw is None:
        dw = _empty(shape, torch.float32, dev, stream)
    rc = lib.mm_grouped_matmul_backward(pd, px, pw, off, cnt, R, K, N, E, dt,
                                        _arg(out, "out", dev, dys.dtype, (R, K)),
                                        _arg(dw, "dw", dev, torch.float32, shape), pws, nbytes, ps, raw)
    del keep                                    # until the work is enqueued
    L.check(rc, "mm_grouped_matmul_backward")
    return out, dw


# --------------------------------------------- microscaled 4-bit floating point
def _mx4_args(q: dict, name: str, dev: int):
    """(address of codes, of exps, shape of the values) of a 4-bit tensor, checked against each other."""
    codes, C = q["codes"], q["cols"]
    if not isinstance(codes, torch.Tensor) or codes.dim() not in (2, 3):
        raise ValueError(f"codes of {name} must be a CUDA tensor [..., R, bytes]")
    if not isinstance(C, int) or C < 1:
        raise ValueError(f"cols of {name} must be a positive whole number")
    lead, groups = codes.shape[:-1], -(-C // _GROUP)
    rows = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    return (_arg(codes, "codes", dev, torch.uint8, (*lead, groups * (_GROUP // 2))),
            _arg(q["exps"], "exps", dev, torch.uint8, (-(-groups // _WORD), rows, _WORD)), (*lead, C))


def mx4_quantize(x: torch.Tensor, *, rows: Optional[torch.Tensor] = None, out: Optional[dict] = None,
                 stream=None) -> dict:
    """x [R, C], or experts' matrices [E, N, C], in 4-bit floating point with a
    power of two per 32 columns (mm_mx4_quantize): a dict of codes (uint8,
    [..., 16 ceil(C / 32)]), exps (uint8 [ceil(C / 128), rows, 4]) and cols C;
    out: such a dict, whose tensors are written anew.  rows (int32 [1] on the
    device, such as a plan's offsets[-1:]): rows from that one on are left alone."""
    if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
        raise ValueError("x must be [R, C] or [E, N, C]")
    dt, dev, raw = _begin(x, "x", x.dim(), stream)
    shape = x.shape
    lead, C = shape[:-1], shape[-1]
    if C < 1:
        raise ValueError("x must have columns")
    R = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    px, pr = _arg(x, "x", dev, x.dtype, shape), _rows_arg(rows, dev)
    if out is None:
        groups = -(-C // _GROUP)
        codes = _empty((*lead, groups * (_GROUP // 2)), torch.uint8, dev, stream)
        exps = _empty((-(-groups // _WORD), R, _WORD), torch.uint8, dev, stream)
        out = {"codes": codes, "exps": exps, "cols": C}
        pc, pe = codes.data_ptr(), exps.data_ptr()
    else:
        pc, pe, held = _mx4_args(out, "out", dev)
        if held != shape:
            raise ValueError(f"out holds {list(held)}, x is {list(shape)}")
    rc = L.load().mm_mx4_quantize(px, R, C, dt, pr, pc, pe, raw)
    L.check(rc, "mm_mx4_quantize")
    return out


def mx4_dequantize(q: dict, dtype: torch.dtype = torch.bfloat16, *, rows: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values that a 4-bit tensor stands for (mm_mx4_dequantize), in
    `dtype`; rows as in mx4_quantize."""
    dev, raw = _device(q["codes"], "codes of q", stream)
    pc, pe, shape = _mx4_args(q, "q", dev)
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {dtype}")
    if out is None:
        out = _empty(shape, dtype, dev, stream)
    R = shape[0] if len(shape) == 2 else shape[0] * shape[1]
    rc = L.load().mm_mx4_dequantize(pc, pe, R, shape[-1], dt, _rows_arg(rows, dev),
                                    _arg(out, "out", dev, dtype, shape), raw)
    L.check(rc, "mm_mx4_dequantize")
    return out


def mx4_matmul_workspace_bytes(rows: int, K: int, N: int, E: int, x_in_4_bits: bool) -> int:
    return int(L.load().mm_mx4_matmul_workspace_bytes(rows, K, N, E, x_in_4_bits))


def mx4_matmul(x: Union[torch.Tensor, dict], w: dict, plan: Optional[dict] = None, *,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               status_workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """grouped_matmul with weights in 4 bits (mm_mx4_matmul): x is bf16 [R, K]
    or mx4_quantize of it, w mx4_quantize of [E, N, K] ([N, K] without a plan);
    ys [R, N] is bf16.  The gradient of x is grouped_matmul_backward's with
    mx4_dequantize(w)."""
    four = isinstance(x, dict)
    if four:
        lead = x["codes"]
        if not isinstance(lead, torch.Tensor) or lead.dim() != 2:
            raise ValueError("codes of x must be [R, bytes]")
    else:
        lead = x
        if isinstance(x, torch.Tensor) and x.is_cuda and x.dtype != torch.bfloat16:
            raise ValueError(f"x must be torch.bfloat16 or a 4-bit dict, got {x.dtype}")
    dev, raw = _device(lead, "x", stream)
    if four:
        px, pxe, (R, K) = _mx4_args(x, "x", dev)
    else:
        if x.dim() != 2:
            raise ValueError(f"x must have 2 dimensions, got {tuple(x.shape)}")
        R, K = x.shape
        px, pxe = _arg(x, "x", dev, torch.bfloat16, (R, K)), None
    off, cnt, E = _plan_args(plan, dev)
    pw, pwe, wshape = _mx4_args(w, "w", dev)
    N = _weight_rows(wshape, plan, "w")
    if wshape != _weight_shape(E, plan is not None, N, K):
        raise ValueError(f"w must be {list(_weight_shape(E, plan is not None, N, K))}, got {list(wshape)}")
    lib = L.load()
    need = _need("mm_mx4_matmul_workspace_bytes", dev, R, K, N, E, four)
    ps = _status_arg(status_workspace, dev)
    pws, nbytes, keep = _scratch(workspace, need, dev, stream, "mx4_matmul")
    if out is None:
        out = _empty((R, N), torch.bfloat16, dev, stream)
    rc = lib.mm_mx4_matmul(px, pxe, pw, pwe, off, cnt, R, K, N, E,
                           _arg(out, "out", dev, torch.bfloat16, (R, N)), pws, nbytes, ps, raw)
    del keep                                    # until the work is enqueued
    L.check(rc, "mm_mx4_matmul")
    return out
