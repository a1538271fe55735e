"""Rows as 8-bit integers: moe_quantize_i8 and moe_dequantize_i8, activation checkpoints
(moe_swiglu_restore_i8) and the products grouped by expert (moe_grouped_gemm_i8 and the SwiGLU expert
FFN moe_grouped_ffn_fwd_i8).  The C entry points and the formulas are in include/moe.h."""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import torch

from . import (MOE_BF16, MOE_F32, _arg, _check, _cuda_device, _cuda_stream, _device, _dtype_code, _int32,
               _into, _raw_stream, _row_type, _shape2, _work, lib)


def moe_quantize_i8(src: torch.Tensor, group: Optional[int] = None, nrows: Optional[torch.Tensor] = None,
                    out: Optional[Dict[str, torch.Tensor]] = None):
    """int8 codes of the rows of src [..., cols] (bf16 or fp32; expert weights [E,N,K] too) with a scale
    for each row, or for each group of 32 to 512 neighbouring columns.  nrows: int32 device tensor whose
    first element bounds the rows written.  Returns (q int8 like src, scale fp32 [...] or
    [..., cols / group])."""
    dt, d, i8, f32 = src.dtype, src.get_device(), torch.int8, torch.float32
    o = out or {}
    q, scale = o.get("q"), o.get("scale")
    if q is not None and scale is not None and nrows is None and src.dim() == 2:
        rows, cols = src.shape
        g = cols if group is None else group
        if (d >= 0 and d == _cuda_device() and not (rows | cols | g) >> 31 and g > 0
                and (dt is torch.bfloat16 or dt is f32) and src.is_contiguous()
                and q.dtype is i8 and q.get_device() == d and q.shape == src.shape and q.is_contiguous()
                and scale.dtype is f32 and scale.get_device() == d and scale.is_contiguous()
                and scale.shape == ((rows,) if group is None else (rows, cols // g))):
            rc = lib.moe_quantize_i8(src.data_ptr(), rows, cols, g,
                                     MOE_BF16 if dt is torch.bfloat16 else MOE_F32, None, q.data_ptr(),
                                     scale.data_ptr(), _cuda_stream(d))
            if rc != 0:
                _check(rc, "moe_quantize_i8")
            return q, scale
    dev = _device(src)
    if src.dim() < 2:
        raise ValueError(f"src must have rows, got shape {tuple(src.shape)}")
    dt = _row_type(src, "src")
    lead, cols = tuple(src.shape[:-1]), src.shape[-1]
    rows = 1
    for n in lead:
        rows *= n
    g = cols if group is None else group
    _int32(rows=rows, cols=cols, group=g)
    if g <= 0 or (cols > 0 and cols % g):
        raise ValueError(f"group={g} must divide the {cols} columns")
    o = {"q": q, "scale": scale}
    nr = _bound(nrows, dev)
    _check(lib.moe_quantize_i8(_arg(src, "src", dt, src.shape, dev), rows, cols, g, _dtype_code(src), nr,
                               _into(o, "q", tuple(src.shape), i8, dev),
                               _into(o, "scale", lead if group is None else lead + (cols // g,), f32, dev),
                               _raw_stream(dev)), "moe_quantize_i8")
    return o["q"], o["scale"]


def _codes(q: torch.Tensor, scale: torch.Tensor, dev):
    """Checked pointers of code rows [rows, cols] with scales [rows] or [rows, groups], and the group."""
    rows, cols = _shape2(q, "q")
    if scale.dim() == 1:
        groups, shape = 1, (rows,)
    else:
        groups = _shape2(scale, "scale")[1]
        shape = (rows, groups)
    if groups < 1 or cols % groups:
        raise ValueError(f"scale has {groups} groups for {cols} columns")
    _int32(rows=rows, cols=cols)
    return (_arg(q, "q", torch.int8, (rows, cols), dev), _arg(scale, "scale", torch.float32, shape, dev),
            rows, cols, cols // groups)


def _bound(nrows: Optional[torch.Tensor], dev) -> Optional[int]:
    if nrows is None:
        return None
    if nrows.dtype != torch.int32 or nrows.device != dev or nrows.numel() < 1:
        raise ValueError(f"nrows must be a non-empty int32 tensor on {dev}")
    return nrows.data_ptr()


def _type_code(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return MOE_BF16
    if dtype == torch.float32:
        return MOE_F32
    raise ValueError(f"dtype must be bf16 or fp32, got {dtype}")


def moe_dequantize_i8(q: torch.Tensor, scale: torch.Tensor, dtype: torch.dtype,
                      src_row: Optional[torch.Tensor] = None, nrows: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None):
    """The values of code rows q [src_rows, cols] with scale [src_rows] or [src_rows, groups]; with src_row
    [rows] int32 row r is that of code row src_row[r].  Returns [rows, cols] of dtype."""
    dev = _device(q)
    qp, sp, src_rows, cols, group = _codes(q, scale, dev)
    rows = src_rows if src_row is None else src_row.numel()
    _int32(rows=rows)
    o = {"out": out}
    _check(lib.moe_dequantize_i8(qp, sp, _arg(src_row, "src_row", torch.int32, (rows,), dev, optional=True),
                                 rows, src_rows, cols, group, _type_code(dtype), _bound(nrows, dev),
                                 _into(o, "out", (rows, cols), dtype, dev), _raw_stream(dev)),
           "moe_dequantize_i8")
    return o["out"]


def moe_swiglu_restore_i8(q: torch.Tensor, scale: torch.Tensor, dtype: torch.dtype,
                          nrows: Optional[torch.Tensor] = None,
                          out: Optional[Dict[str, torch.Tensor]] = None):
    """gu [rows, 2I] and h_perm = SiLU(g) * u [rows, I] of dtype, from the codes q [rows, 2I] of a forward's
    gu with scale [rows] or [rows, groups].  Returns dict gu, h_perm."""
    d, dt = q.get_device(), dtype
    o = dict(out) if out else {}
    gu, h = o.get("gu"), o.get("h_perm")
    if gu is not None and h is not None and nrows is None and q.dim() == 2 and scale.dim() == 2:
        rows, cols = q.shape
        groups = scale.shape[1]
        if (d >= 0 and d == _cuda_device() and not (rows | cols | groups) >> 31 and groups > 0
                and cols % (2 * groups) == 0 and (dt is torch.bfloat16 or dt is torch.float32)
                and q.dtype is torch.int8 and q.is_contiguous()
                and scale.dtype is torch.float32 and scale.get_device() == d and scale.shape[0] == rows
                and scale.is_contiguous()
                and gu.dtype is dt and gu.get_device() == d and gu.shape == q.shape and gu.is_contiguous()
                and h.dtype is dt and h.get_device() == d and h.shape == (rows, cols // 2)
                and h.is_contiguous()):
            rc = lib.moe_swiglu_restore_i8(q.data_ptr(), scale.data_ptr(), rows, cols // 2, cols // groups,
                                           MOE_BF16 if dt is torch.bfloat16 else MOE_F32, None,
                                           gu.data_ptr(), h.data_ptr(), _cuda_stream(d))
            if rc != 0:
                _check(rc, "moe_swiglu_restore_i8")
            return o
    dev = _device(q)
    qp, sp, rows, cols, group = _codes(q, scale, dev)
    if cols % 2:
        raise ValueError(f"q holds gate and up: an even number of columns, got {cols}")
    _check(lib.moe_swiglu_restore_i8(qp, sp, rows, cols // 2, group, _type_code(dtype), _bound(nrows, dev),
                                     _into(o, "gu", (rows, cols), dtype, dev),
                                     _into(o, "h_perm", (rows, cols // 2), dtype, dev), _raw_stream(dev)),
           "moe_swiglu_restore_i8")
    return o


def moe_grouped_gemm_i8(x_q: torch.Tensor, x_scale: torch.Tensor, src_row: Optional[torch.Tensor],
                        offsets: torch.Tensor, w_q: torch.Tensor, w_scale: torch.Tensor,
                        out: Optional[torch.Tensor] = None):
    """Product of int8 rows with int8 weights w_q [E_l,N,K], grouped by expert: row r of expert e
    (offsets [E_l+1] int32) is x_q[src_row[r]] (src_row None: x_q[r]); scales x_scale [x_rows] and
    w_scale [E_l,N] fp32.  Returns y [R_cap,N] bf16, rows past offsets[E_l] not written."""
    i8, i32, f32, d = torch.int8, torch.int32, torch.float32, x_q.get_device()
    if out is not None and src_row is not None and x_q.dim() == 2 and w_q.dim() == 3:
        x_rows, K = x_q.shape
        E_l, N = w_q.shape[0], w_q.shape[1]
        R_cap = src_row.numel()
        if (d >= 0 and d == _cuda_device() and not (x_rows | K | E_l | N | R_cap) >> 31
                and x_q.dtype is i8 and x_q.is_contiguous()
                and x_scale.dtype is f32 and x_scale.get_device() == d and x_scale.shape == (x_rows,)
                and x_scale.is_contiguous()
                and src_row.dtype is i32 and src_row.get_device() == d and src_row.dim() == 1
                and src_row.is_contiguous()
                and offsets.dtype is i32 and offsets.get_device() == d and offsets.shape == (E_l + 1,)
                and offsets.is_contiguous()
                and w_q.dtype is i8 and w_q.get_device() == d and w_q.shape[2] == K and w_q.is_contiguous()
                and w_scale.dtype is f32 and w_scale.get_device() == d and w_scale.shape == (E_l, N)
                and w_scale.is_contiguous()
                and out.dtype is torch.bfloat16 and out.get_device() == d and out.shape == (R_cap, N)
                and out.is_contiguous()):
            rc = lib.moe_grouped_gemm_i8(x_q.data_ptr(), x_scale.data_ptr(), src_row.data_ptr(),
                                         offsets.data_ptr(), E_l, R_cap, x_rows, K, N, w_q.data_ptr(),
                                         w_scale.data_ptr(), out.data_ptr(), _cuda_stream(d))
            if rc != 0:
                _check(rc, "moe_grouped_gemm_i8")
            return out
    dev = _device(x_q)
    x_rows, K = _shape2(x_q, "x_q")
    if w_q.dim() != 3:
        raise ValueError(f"w_q must be [E_l, N, K], got shape {tuple(w_q.shape)}")
    E_l, N = w_q.shape[:2]
    R_cap = x_rows if src_row is None else src_row.numel()
    _int32(x_rows=x_rows, K=K, E_l=E_l, N=N, R_cap=R_cap)
    o = {"y": out}
    _check(lib.moe_grouped_gemm_i8(
        _arg(x_q, "x_q", i8, (x_rows, K), dev), _arg(x_scale, "x_scale", f32, (x_rows,), dev),
        _arg(src_row, "src_row", i32, (R_cap,), dev, optional=True),
        _arg(offsets, "offsets", i32, (E_l + 1,), dev), E_l, R_cap, x_rows, K, N,
        _arg(w_q, "w_q", i8, (E_l, N, K), dev), _arg(w_scale, "w_scale", f32, (E_l, N), dev),
        _into(o, "y", (R_cap, N), torch.bfloat16, dev), _raw_stream(dev)), "moe_grouped_gemm_i8")
    return o["y"]


def _ffn_i8_ws_bytes(R_cap: int, I: int) -> int:
    nb = lib.moe_ffn_i8_ws_bytes(R_cap, I)
    if nb < 0:
        _check(int(nb), "moe_ffn_i8_ws_bytes")
    return int(nb)


def moe_grouped_ffn_fwd_i8(x_q: torch.Tensor, x_scale: torch.Tensor, src_row: Optional[torch.Tensor],
                           offsets: torch.Tensor, wg: Tuple[torch.Tensor, torch.Tensor],
                           wu: Tuple[torch.Tensor, torch.Tensor], wd: Tuple[torch.Tensor, torch.Tensor],
                           ws: Optional[torch.Tensor] = None, out: Optional[Dict[str, torch.Tensor]] = None):
    """Grouped SwiGLU FFN forward on int8 codes: rows as in moe_grouped_gemm_i8, wg / wu / wd = (codes int8
    [E_l,I,H] / [E_l,H,I], channel scales fp32 [E_l,I] / [E_l,H]) of moe_quantize_i8.  Returns dict h_perm
    [R_cap,I], y_perm [R_cap,H] (bf16) and the workspace ws used."""
    i8, i32, f32, bf, d = torch.int8, torch.int32, torch.float32, torch.bfloat16, x_q.get_device()
    o = dict(out) if out else {}
    (gq, gs), (uq, us), (dq, ds) = wg, wu, wd
    h, y = o.get("h_perm"), o.get("y_perm")
    if (h is not None and y is not None and ws is not None and src_row is not None and x_q.dim() == 2
            and gq.dim() == 3):
        x_rows, H = x_q.shape
        E_l, I = gq.shape[0], gq.shape[1]
        R_cap = src_row.numel()
        if (d >= 0 and d == _cuda_device() and not (x_rows | H | E_l | I | R_cap) >> 31
                and x_q.dtype is i8 and x_q.is_contiguous()
                and x_scale.dtype is f32 and x_scale.get_device() == d and x_scale.shape == (x_rows,)
                and x_scale.is_contiguous()
                and src_row.dtype is i32 and src_row.get_device() == d and src_row.dim() == 1
                and src_row.is_contiguous()
                and offsets.dtype is i32 and offsets.get_device() == d and offsets.shape == (E_l + 1,)
                and offsets.is_contiguous()
                and gq.dtype is i8 and gq.get_device() == d and gq.shape[2] == H and gq.is_contiguous()
                and uq.dtype is i8 and uq.get_device() == d and uq.shape == gq.shape and uq.is_contiguous()
                and dq.dtype is i8 and dq.get_device() == d and dq.shape == (E_l, H, I)
                and dq.is_contiguous()
                and gs.dtype is f32 and gs.get_device() == d and gs.shape == (E_l, I) and gs.is_contiguous()
                and us.dtype is f32 and us.get_device() == d and us.shape == (E_l, I) and us.is_contiguous()
                and ds.dtype is f32 and ds.get_device() == d and ds.shape == (E_l, H) and ds.is_contiguous()
                and h.dtype is bf and h.get_device() == d and h.shape == (R_cap, I) and h.is_contiguous()
                and y.dtype is bf and y.get_device() == d and y.shape == (R_cap, H) and y.is_contiguous()
                and ws.get_device() == d and ws.is_contiguous()):
            rc = lib.moe_grouped_ffn_fwd_i8(
                x_q.data_ptr(), x_scale.data_ptr(), src_row.data_ptr(), offsets.data_ptr(), E_l, R_cap,
                x_rows, H, I, gq.data_ptr(), gs.data_ptr(), uq.data_ptr(), us.data_ptr(), dq.data_ptr(),
                ds.data_ptr(), h.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.nbytes, _cuda_stream(d))
            if rc != 0:
                _check(rc, "moe_grouped_ffn_fwd_i8")
            o["ws"] = ws
            return o
    dev = _device(x_q)
    x_rows, H = _shape2(x_q, "x_q")
    if gq.dim() != 3:
        raise ValueError(f"the codes of wg must be [E_l, I, H], got shape {tuple(gq.shape)}")
    E_l, I = gq.shape[:2]
    R_cap = x_rows if src_row is None else src_row.numel()
    _int32(x_rows=x_rows, H=H, E_l=E_l, I=I, R_cap=R_cap)
    a = [_arg(x_q, "x_q", i8, (x_rows, H), dev), _arg(x_scale, "x_scale", f32, (x_rows,), dev),
         _arg(src_row, "src_row", i32, (R_cap,), dev, optional=True),
         _arg(offsets, "offsets", i32, (E_l + 1,), dev)]
    w = []
    for name, (q, s), n, k in (("wg", wg, I, H), ("wu", wu, I, H), ("wd", wd, H, I)):
        w += [_arg(q, f"the codes of {name}", i8, (E_l, n, k), dev),
              _arg(s, f"the scales of {name}", f32, (E_l, n), dev)]
    o["ws"] = _work(_ffn_i8_ws_bytes(R_cap, I), dev, ws)
    _check(lib.moe_grouped_ffn_fwd_i8(
        *a, E_l, R_cap, x_rows, H, I, *w, _into(o, "h_perm", (R_cap, I), bf, dev),
        _into(o, "y_perm", (R_cap, H), bf, dev), None if o["ws"] is None else o["ws"].data_ptr(),
        0 if o["ws"] is None else o["ws"].nbytes, _raw_stream(dev)), "moe_grouped_ffn_fwd_i8")
    return o
