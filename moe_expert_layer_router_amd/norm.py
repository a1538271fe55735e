"""RMS norms around the layer: moe_norm (the residual update and the norm before it) and
moe_combine_norm (the combine with the norm after it, a gate and the scaled residual), each with its
backward.  The C entry points and the formulas are in include/moe.h."""
from __future__ import annotations

from typing import Dict, Optional

import torch

from . import (MOE_BF16, MOE_F32, _arg, _check, _cuda_device, _cuda_stream, _device, _dtype_code, _int32,
               _into, _raw_stream, _row_type, _shape2, _work, lib)

GATE_NONE, GATE_TOKEN, GATE_FULL = range(3)


def _norm_ws_bytes(H: int) -> int:
    nb = lib.moe_norm_ws_bytes(H)
    if nb < 0:
        _check(int(nb), "moe_norm_ws_bytes")
    return int(nb)


def moe_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, delta: Optional[torch.Tensor] = None,
             out: Optional[Dict[str, torch.Tensor]] = None):
    """r = x + delta (delta None: r is x) and n = r / sqrt(mean r^2 + eps) * weight, for x [T,H] and
    weight [H] fp32.  Returns dict n and r (out["r"] may be x or delta: an update in place)."""
    o = dict(out) if out else {}
    dt, f32, d = x.dtype, torch.float32, x.get_device()
    n, r = o.get("n"), o.get("r")
    # a call that gives every tensor, checked in one expression
    if n is not None and x.dim() == 2 and (delta is None or r is not None):
        T, H = x.shape
        if (d >= 0 and d == _cuda_device() and not (T | H) >> 31
                and (dt is torch.bfloat16 or dt is f32) and x.is_contiguous()
                and weight.dtype is f32 and weight.get_device() == d and weight.shape == (H,)
                and weight.is_contiguous()
                and n.dtype is dt and n.get_device() == d and n.shape == x.shape and n.is_contiguous()
                and (delta is None or delta.dtype is dt and delta.get_device() == d
                     and delta.shape == x.shape and delta.is_contiguous()
                     and r.dtype is dt and r.get_device() == d and r.shape == x.shape
                     and r.is_contiguous())):
            rc = lib.moe_norm(x.data_ptr(), None if delta is None else delta.data_ptr(), weight.data_ptr(),
                              eps, T, H, MOE_BF16 if dt is torch.bfloat16 else MOE_F32,
                              None if delta is None else r.data_ptr(), n.data_ptr(), _cuda_stream(d))
            if rc != 0:
                _check(rc, "moe_norm")
            if delta is None:
                o["r"] = x
            return o
    dev = _device(x)
    T, H = _shape2(x, "x")
    _int32(T=T, H=H)
    dt = _row_type(x, "x")
    a = [_arg(x, "x", dt, (T, H), dev), _arg(delta, "delta", dt, (T, H), dev, optional=True),
         _arg(weight, "weight", f32, (H,), dev)]
    if delta is None:
        o["r"] = x
    rp = None if delta is None else _into(o, "r", (T, H), dt, dev)
    _check(lib.moe_norm(*a, eps, T, H, _dtype_code(x), rp, _into(o, "n", (T, H), dt, dev), _raw_stream(dev)),
           "moe_norm")
    return o


def moe_norm_bwd(dn: torch.Tensor, r: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 dr: Optional[torch.Tensor] = None, dr_scale: float = 1.0, accumulate: bool = False,
                 ws: Optional[torch.Tensor] = None, out: Optional[Dict[str, torch.Tensor]] = None):
    """Backward of moe_norm for the gradient dn of n and (optional) dr_scale * dr of r.  Returns dict dx [T,H] (of
    x and of delta), dweight [H] fp32 (added to with accumulate=True) and the workspace ws used."""
    o = dict(out) if out else {}
    dt, f32, d = dn.dtype, torch.float32, dn.get_device()
    dx, dw = o.get("dx"), o.get("dweight")
    if dx is not None and dw is not None and ws is not None and dn.dim() == 2:
        T, H = dn.shape
        if (d >= 0 and d == _cuda_device() and not (T | H) >> 31
                and (dt is torch.bfloat16 or dt is f32) and dn.is_contiguous()
                and r.dtype is dt and r.get_device() == d and r.shape == dn.shape and r.is_contiguous()
                and weight.dtype is f32 and weight.get_device() == d and weight.shape == (H,)
                and weight.is_contiguous()
                and (dr is None or dr.dtype is dt and dr.get_device() == d and dr.shape == dn.shape
                     and dr.is_contiguous())
                and dx.dtype is dt and dx.get_device() == d and dx.shape == dn.shape and dx.is_contiguous()
                and dw.dtype is f32 and dw.get_device() == d and dw.shape == (H,) and dw.is_contiguous()
                and ws.get_device() == d and ws.is_contiguous()):
            rc = lib.moe_norm_bwd(dn.data_ptr(), None if dr is None else dr.data_ptr(), dr_scale, r.data_ptr(),
                                  weight.data_ptr(), eps, T, H,
                                  MOE_BF16 if dt is torch.bfloat16 else MOE_F32, dx.data_ptr(),
                                  dw.data_ptr(), 1 if accumulate else 0, ws.data_ptr(), ws.nbytes,
                                  _cuda_stream(d))
            if rc != 0:
                _check(rc, "moe_norm_bwd")
            o["ws"] = ws
            return o
    dev = _device(dn)
    T, H = _shape2(dn, "dn")
    _int32(T=T, H=H)
    dt = _row_type(dn, "dn")
    a = [_arg(dn, "dn", dt, (T, H), dev), _arg(dr, "dr", dt, (T, H), dev, optional=True), dr_scale,
         _arg(r, "r", dt, (T, H), dev), _arg(weight, "weight", f32, (H,), dev)]
    if accumulate and dw is None:
        raise ValueError("accumulate=True needs out with dweight")
    o["ws"] = _work(_norm_ws_bytes(H), dev, ws)
    _check(lib.moe_norm_bwd(*a, eps, T, H, _dtype_code(dn), _into(o, "dx", (T, H), dt, dev),
                            _into(o, "dweight", (H,), f32, dev), 1 if accumulate else 0,
                            o["ws"].data_ptr(), o["ws"].nbytes, _raw_stream(dev)), "moe_norm_bwd")
    return o


def _gate_kind(gate: Optional[torch.Tensor]) -> int:
    if gate is None:
        return GATE_NONE
    if gate.dim() not in (1, 2):
        raise ValueError(f"gate must be [T] or [T, H], got shape {tuple(gate.shape)}")
    return GATE_TOKEN if gate.dim() == 1 else GATE_FULL


def _gate_ok(gate: torch.Tensor, dt, d: int, T: int, H: int) -> bool:
    return (gate.get_device() == d and gate.is_contiguous()
            and (gate.dtype is torch.float32 and gate.shape == (T,) or gate.dtype is dt and gate.shape == (T, H)))


def moe_combine_norm(y_perm: torch.Tensor, topk_w: Optional[torch.Tensor], dest_row: torch.Tensor, T: int,
                     weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                     residual_scale: float = 1.0, gate: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None):
    """residual_scale * residual + gate * norm(combine) * weight, for the combine of moe_combine, weight
    [H] fp32 and gate None, [T] fp32 or [T,H] (dtype).  Returns y [T,H] (out may be residual)."""
    dt, f32, d = y_perm.dtype, torch.float32, y_perm.get_device()
    if out is not None and topk_w is not None and y_perm.dim() == 2 and topk_w.dim() == 2:
        H, k = y_perm.shape[1], topk_w.shape[1]
        if (d >= 0 and d == _cuda_device() and not (T | H | k) >> 31
                and (dt is torch.bfloat16 or dt is f32) and y_perm.is_contiguous()
                and topk_w.dtype is f32 and topk_w.get_device() == d and topk_w.shape[0] == T
                and topk_w.is_contiguous()
                and dest_row.dtype is torch.int32 and dest_row.get_device() == d
                and dest_row.shape == (T * k,) and dest_row.is_contiguous()
                and weight.dtype is f32 and weight.get_device() == d and weight.shape == (H,)
                and weight.is_contiguous()
                and (residual is None or residual.dtype is dt and residual.get_device() == d
                     and residual.shape == (T, H) and residual.is_contiguous())
                and (gate is None or _gate_ok(gate, dt, d, T, H))
                and out.dtype is dt and out.get_device() == d and out.shape == (T, H)
                and out.is_contiguous()):
            rc = lib.moe_combine_norm(
                y_perm.data_ptr(), topk_w.data_ptr(), dest_row.data_ptr(),
                None if residual is None else residual.data_ptr(), residual_scale,
                None if gate is None else gate.data_ptr(), 0 if gate is None else gate.dim(),
                weight.data_ptr(), eps, T, H, k, MOE_BF16 if dt is torch.bfloat16 else MOE_F32,
                out.data_ptr(), _cuda_stream(d))
            if rc != 0:
                _check(rc, "moe_combine_norm")
            return out
    dev = _device(y_perm)
    R_cap, H = _shape2(y_perm, "y_perm")
    if T < 0 or (T == 0 and dest_row.numel()) or (T > 0 and dest_row.numel() % T):
        raise ValueError(f"dest_row has {dest_row.numel()} entries, not k for each of {T} tokens")
    k = _shape2(topk_w, "topk_w")[1] if topk_w is not None else max(dest_row.numel() // max(T, 1), 1)
    _int32(T=T, H=H, k=k)
    dt = _row_type(y_perm, "y_perm")
    kind = _gate_kind(gate)
    o = {"y": out}
    a = [_arg(y_perm, "y_perm", dt, (R_cap, H), dev), _arg(topk_w, "topk_w", f32, (T, k), dev, optional=True),
         _arg(dest_row, "dest_row", torch.int32, (T * k,), dev),
         _arg(residual, "residual", dt, (T, H), dev, optional=True)]
    gp = _arg(gate, "gate", f32 if kind == GATE_TOKEN else dt, (T,) if kind == GATE_TOKEN else (T, H), dev,
              optional=True)
    _check(lib.moe_combine_norm(*a, residual_scale, gp, kind, _arg(weight, "weight", f32, (H,), dev), eps, T,
                                H, k, _dtype_code(y_perm), _into(o, "y", (T, H), dt, dev), _raw_stream(dev)),
           "moe_combine_norm")
    return o["y"]


def moe_combine_norm_bwd(dy: torch.Tensor, y_perm: torch.Tensor, topk_w: torch.Tensor,
                         dest_row: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                         gate: Optional[torch.Tensor] = None, accumulate: bool = False,
                         ws: Optional[torch.Tensor] = None, out: Optional[Dict[str, torch.Tensor]] = None):
    """Backward of moe_combine_norm for dy [T,H].  Returns dict dy_perm [R_cap,H], d_topk_w [T,k] fp32,
    dweight [H] fp32 (added to with accumulate=True), dgate (of the gate's shape and type, or None) and
    the workspace ws used.  The residual's gradient is residual_scale * dy."""
    o = dict(out) if out else {}
    dt, f32, d = dy.dtype, torch.float32, dy.get_device()
    dyp, dk, dw, dg = o.get("dy_perm"), o.get("d_topk_w"), o.get("dweight"), o.get("dgate")
    if (dyp is not None and dk is not None and dw is not None and ws is not None
            and (gate is None or dg is not None) and dy.dim() == 2 and y_perm.dim() == 2
            and topk_w.dim() == 2):
        T, H = dy.shape
        k = topk_w.shape[1]
        if (d >= 0 and d == _cuda_device() and not (T | H | k) >> 31
                and (dt is torch.bfloat16 or dt is f32) and dy.is_contiguous()
                and y_perm.dtype is dt and y_perm.get_device() == d and y_perm.shape[1] == H
                and y_perm.is_contiguous()
                and topk_w.dtype is f32 and topk_w.get_device() == d and topk_w.shape[0] == T
                and topk_w.is_contiguous()
                and dest_row.dtype is torch.int32 and dest_row.get_device() == d
                and dest_row.shape == (T * k,) and dest_row.is_contiguous()
                and weight.dtype is f32 and weight.get_device() == d and weight.shape == (H,)
                and weight.is_contiguous()
                and (gate is None or _gate_ok(gate, dt, d, T, H) and dg.dtype is gate.dtype
                     and dg.get_device() == d and dg.shape == gate.shape and dg.is_contiguous())
                and dyp.dtype is dt and dyp.get_device() == d and dyp.shape == y_perm.shape
                and dyp.is_contiguous()
                and dk.dtype is f32 and dk.get_device() == d and dk.shape == topk_w.shape
                and dk.is_contiguous()
                and dw.dtype is f32 and dw.get_device() == d and dw.shape == (H,) and dw.is_contiguous()
                and ws.get_device() == d and ws.is_contiguous()):
            rc = lib.moe_combine_norm_bwd(
                dy.data_ptr(), y_perm.data_ptr(), topk_w.data_ptr(), dest_row.data_ptr(),
                None if gate is None else gate.data_ptr(), 0 if gate is None else gate.dim(),
                weight.data_ptr(), eps, T, H, k, MOE_BF16 if dt is torch.bfloat16 else MOE_F32,
                dyp.data_ptr(), dk.data_ptr(), None if gate is None else dg.data_ptr(), dw.data_ptr(),
                1 if accumulate else 0, ws.data_ptr(), ws.nbytes, _cuda_stream(d))
            if rc != 0:
                _check(rc, "moe_combine_norm_bwd")
            if gate is None:
                o["dgate"] = None
            o["ws"] = ws
            return o
    dev = _device(dy)
    T, H = _shape2(dy, "dy")
    k, R_cap = _shape2(topk_w, "topk_w")[1], _shape2(y_perm, "y_perm")[0]
    _int32(T=T, H=H, k=k)
    dt = _row_type(dy, "dy")
    kind = _gate_kind(gate)
    gate_as = (f32, (T,)) if kind == GATE_TOKEN else (dt, (T, H))
    a = [_arg(dy, "dy", dt, (T, H), dev), _arg(y_perm, "y_perm", dt, (R_cap, H), dev),
         _arg(topk_w, "topk_w", f32, (T, k), dev), _arg(dest_row, "dest_row", torch.int32, (T * k,), dev),
         _arg(gate, "gate", *gate_as, dev, optional=True)]
    wp = _arg(weight, "weight", f32, (H,), dev)
    if accumulate and dw is None:
        raise ValueError("accumulate=True needs out with dweight")
    gp = None
    if kind == GATE_NONE:
        o["dgate"] = None
    else:
        gp = _into(o, "dgate", gate_as[1], gate_as[0], dev)
    o["ws"] = _work(_norm_ws_bytes(H), dev, ws)
    _check(lib.moe_combine_norm_bwd(*a, kind, wp, eps, T, H, k, _dtype_code(dy),
                                    _into(o, "dy_perm", (R_cap, H), dt, dev),
                                    _into(o, "d_topk_w", (T, k), f32, dev), gp,
                                    _into(o, "dweight", (H,), f32, dev), 1 if accumulate else 0,
                                    o["ws"].data_ptr(), o["ws"].nbytes, _raw_stream(dev)),
           "moe_combine_norm_bwd")
    return o
