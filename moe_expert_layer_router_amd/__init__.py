"""Python binding of the gfx950 MoE expert layer library (libmoe.so).

Argument marshalling only: every step of the layer runs in the HIP kernels
behind the C ABI declared in include/moe.h.  PyTorch provides device memory
(outputs and workspaces are torch tensors) and the stream (the current torch
stream).  There is no fallback: importing this package fails when the built
library is missing, and every call raises MoEError when the library reports
an error.

Functions keep the C names (moe_route, moe_permute, moe_grouped_ffn_fwd and its
gathering form moe_grouped_ffn_fwd_gather, moe_combine, moe_combine_bwd, moe_grouped_ffn_bwd, moe_route_bwd, and the FP8
forward: moe_quantize_fp8, moe_grouped_ffn_fwd_fp8; data gradients:
moe_quantize_fp8_t, moe_grouped_ffn_dgrad_fp8; both weight layouts at once:
moe_quantize_fp8_w; weight gradients:
moe_quantize_fp8_group_t, moe_grouped_ffn_wgrad_fp8, and its two halves
moe_grouped_ffn_wgrad_fp8_begin / _end; around the layer: the router's
auxiliary losses moe_balance_loss / _bwd with moe_route_bwd_add, and the combine
with dropout moe_combine_dropout / _bwd, and low-rank adapters moe_adapter_fwd /
_bwd with moe_adapter_rows and moe_grouped_ffn_fwd_adapter) and return
freshly allocated torch tensors; each also accepts preallocated outputs via
``out=`` dictionaries so that steady-state loops allocate nothing.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Dict, Optional

import torch  # loads torch's HIP runtime first, so libmoe binds to the same one

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_F32, MOE_BF16, MOE_FP8 = 0, 1, 2
(MOE_OP_ROUTE, MOE_OP_PERMUTE, MOE_OP_FFN_FWD, MOE_OP_FFN_BWD, MOE_OP_ROUTE_BWD,
 MOE_OP_COMBINE_DX, MOE_OP_FFN_FWD_FP8, MOE_OP_FFN_DGRAD_FP8, MOE_OP_FFN_WGRAD_FP8,
 MOE_OP_QUANTIZE_W_FP8) = range(10)
ABI_VERSION = 10


class MoEError(RuntimeError):
    pass


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run __graft_entry__.build() (hipcc --offload-arch=gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    F32, F64 = ctypes.c_float, ctypes.c_double
    sig = {
        "moe_abi_version": ([], I32),
        "moe_last_error": ([], ctypes.c_char_p),
        "moe_workspace_bytes": ([I32] * 9, I64),
        "moe_route": ([P, P, P, I32, I32, I32, I32, I32, P, P, P, P, SZ, P], I32),
        "moe_route_from_logits": ([P, I32, I32, I32, P, P, P], I32),
        "moe_permute": ([P, P, I32, I32, I32, I32, I32, I32, I32, P, P, P, P, P, P, SZ, P], I32),
        "moe_grouped_ffn_fwd": ([P, P, I32, I32, I32, I32, P, P, P, I32, P, P, P, P, SZ, P], I32),
        "moe_grouped_ffn_fwd_noalloc": ([P, P, I32, I32, I32, I32, P, P, P, I32, P, P, P, P], I32),
        "moe_grouped_ffn_fwd_gather": ([P, P, P, I32, I32, I32, I32, I32, P, P, P, I32, P, P, P, P, SZ,
                                        P], I32),
        "moe_combine": ([P, P, P, P, I32, I32, I32, I32, P, P], I32),
        "moe_combine_bwd": ([P, P, P, P, I32, I32, I32, I32, P, P, P], I32),
        "moe_combine_dx": ([P, P, P, P, P, P, I32, I32, I32, I32, I32, P, P, SZ, P], I32),
        "moe_combine_dx_t": ([P, P, P, P, P, P, I32, I32, I32, I32, I32, P, P], I32),
        "moe_router_weight_t": ([P, I32, I32, I32, P, P], I32),
        "moe_grouped_ffn_bwd": ([P, P, P, P, P, I32, I32, I32, I32, P, P, P, I32, P, P, P, P, I32,
                                 P, SZ, P], I32),
        "moe_grouped_ffn_bwd_split": ([P, P, P, P, P, I32, I32, I32, I32, P, P, P, I32, P, P, P, P,
                                       I32, P, SZ, P, P], I32),
        "moe_route_bwd": ([P, P, P, P, P, I32, I32, I32, I32, I32, P, P, P, P, SZ, P], I32),
        "moe_quantize_fp8": ([P, I32, I32, I32, P, P, P, P], I32),
        "moe_quantize_fp8_t": ([P, P, I32, I32, I32, I32, P, P, P], I32),
        "moe_grouped_ffn_dgrad_fp8": ([P, P, P, P, I32, I32, I32, I32, P, P, P, P, P, P, P, SZ, P], I32),
        "moe_grouped_ffn_fwd_fp8_gather": ([P, P, P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, P, P,
                                            P, P, SZ, P], I32),
        "moe_grouped_ffn_fwd_fp8": ([P, P, P, P, I32, I32, I32, I32, P, P, P, P, P, P, P, P, P, P,
                                     SZ, P], I32),
        "moe_quantize_fp8_group_t": ([P, P, I32, P, I32, I32, P, I32, P, P, P], I32),
        "moe_quantize_fp8_w": ([P, P, I32, I32, I32, I32, P, P, P, P, P, P, P, SZ, P], I32),
        "moe_grouped_ffn_wgrad_fp8": ([P, P, P, P, P, P, I32, I32, I32, I32, P, P, P, I32, P, SZ, P],
                                      I32),
        "moe_grouped_ffn_wgrad_fp8_begin": ([P, P, P, P, P, I32, I32, I32, I32, P, I32, P, SZ, P], I32),
        "moe_grouped_ffn_wgrad_fp8_end": ([P, P, I32, I32, I32, I32, P, P, P, I32, P, SZ, P], I32),
        "moe_route_bwd_add": ([P, P, P, P, P, P, I32, I32, I32, I32, I32, P, P, P, P, SZ, P], I32),
        "moe_balance_ws_bytes": ([I32] * 3, I64),
        "moe_balance_loss": ([P, P, P, P, I32, I32, I32, I32, F32, F32, P, P, P, P, P, P, SZ, P], I32),
        "moe_balance_loss_bwd": ([P, P, P, P, P, P, P, I32, I32, I32, I32, F32, F32, I32, P, P], I32),
        "moe_combine_dropout": ([P, P, P, P, F64, P, I32, I32, I32, I32, P, P], I32),
        "moe_combine_dropout_bwd": ([P, P, P, P, F64, P, I32, I32, I32, I32, P, P, P], I32),
        "moe_adapter_fwd": ([P] * 6 + [I32] * 9 + [P, P, P], I32),
        "moe_adapter_ws_bytes": ([I32] * 6, I64),
        "moe_adapter_bwd": ([P] * 8 + [I32] * 10 + [P, P, P, I32, P, SZ, P], I32),
        "moe_grouped_ffn_fwd_adapter": ([P] * 4 + [I32] * 5 + [P] * 10 + [I32] * 3 + [P, P, P, P, SZ, P],
                                        I32),
        "moe_adapter_rows": ([P, P, P, I32, I32, I32, I32, P, P], I32),
        "moe_profile_kernel": ([I32, ctypes.POINTER(P), ctypes.POINTER(P), I32], I32),
        "moe_profile_recorded": ([], I32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if lib.moe_abi_version() != ABI_VERSION:
        raise ImportError(f"libmoe ABI {lib.moe_abi_version()} != binding ABI {ABI_VERSION}")
    return lib


lib = _load()


def hip_runtimes_mapped():
    """Paths of every libamdhip64 mapped into this process (should be one)."""
    try:
        with open("/proc/self/maps") as f:
            return sorted({ln.split()[-1] for ln in f if "libamdhip64" in ln})
    except OSError:
        return []


def _check(rc: int, what: str):
    if rc != 0:
        raise MoEError(f"{what} failed ({rc}): {lib.moe_last_error().decode()}")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.uint8:  # E4M3 codes
        return MOE_FP8
    raise ValueError(f"unsupported dtype {t.dtype}")


def workspace_bytes(op: int, T: int, H: int, I: int, E: int, k: int, e_lo: int, e_hi: int,
                    dtype: int) -> int:
    n = lib.moe_workspace_bytes(op, T, H, I, E, k, e_lo, e_hi, dtype)
    if n < 0:
        _check(int(n), "moe_workspace_bytes")
    return int(n)


def _ws(nbytes: int, device, ws: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return ws
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError(f"workspace too small: {nbytes} bytes needed")
        return ws
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


# ---------------------------------------------------------------------------
# ABI wrappers
# ---------------------------------------------------------------------------

def moe_route(x: torch.Tensor, w_router: torch.Tensor, k: int, bias: Optional[torch.Tensor] = None,
              want_logits: bool = False, ws: Optional[torch.Tensor] = None,
              out: Optional[Dict[str, torch.Tensor]] = None):
    """Router GEMM + top-k gating.  Returns (topk_idx int32 [T,k], topk_w fp32 [T,k], logits|None)."""
    T, H = x.shape
    E = w_router.shape[1]
    dt = _dtype_code(x)
    out = out or {}
    idx = out.get("topk_idx")
    if idx is None:
        idx = torch.empty((T, k), dtype=torch.int32, device=x.device)
    w = out.get("topk_w")
    if w is None:
        w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    logits = out.get("logits")
    if want_logits and logits is None:
        logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    ws = _ws(workspace_bytes(MOE_OP_ROUTE, T, H, 1, E, k, 0, E, dt), x.device, ws)
    _check(lib.moe_route(_ptr(x), _ptr(w_router), _ptr(bias), T, H, E, k, dt, _ptr(logits),
                         _ptr(idx), _ptr(w), _ptr(ws), _nbytes(ws), _stream()), "moe_route")
    return idx, w, logits


def moe_route_from_logits(logits: torch.Tensor, k: int):
    T, E = logits.shape
    idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(lib.moe_route_from_logits(_ptr(logits), T, E, k, _ptr(idx), _ptr(w), _stream()),
           "moe_route_from_logits")
    return idx, w


def moe_permute(x: torch.Tensor, topk_idx: torch.Tensor, E: int, e_lo: int, e_hi: int,
                ws: Optional[torch.Tensor] = None, out: Optional[Dict[str, torch.Tensor]] = None,
                copy_rows: bool = True):
    """Group routed rows by expert.  Returns dict counts, offsets, dest_row, src_row, x_perm
    (x_perm None with copy_rows=False: the maps alone, for moe_grouped_ffn_fwd_gather)."""
    T, H = x.shape
    k = topk_idx.shape[1]
    dt = _dtype_code(x)
    E_l = e_hi - e_lo
    dev = x.device
    o = dict(out or {})
    o.setdefault("counts", torch.empty(E_l, dtype=torch.int32, device=dev))
    o.setdefault("offsets", torch.empty(E_l + 1, dtype=torch.int32, device=dev))
    o.setdefault("dest_row", torch.empty(T * k, dtype=torch.int32, device=dev))
    o.setdefault("src_row", torch.empty(T * k, dtype=torch.int32, device=dev))
    if copy_rows:
        o.setdefault("x_perm", torch.empty((T * k, H), dtype=x.dtype, device=dev))
    else:
        o["x_perm"] = None
    ws = _ws(workspace_bytes(MOE_OP_PERMUTE, T, H, 1, E, k, e_lo, e_hi, dt), dev, ws)
    _check(lib.moe_permute(_ptr(x), _ptr(topk_idx), T, H, E, k, e_lo, e_hi, dt, _ptr(o["counts"]),
                           _ptr(o["offsets"]), _ptr(o["dest_row"]), _ptr(o["src_row"]),
                           _ptr(o["x_perm"]), _ptr(ws), _nbytes(ws), _stream()), "moe_permute")
    return o


def moe_grouped_ffn_fwd(x_perm: torch.Tensor, offsets: torch.Tensor, w_gate: torch.Tensor,
                        w_up: torch.Tensor, w_down: torch.Tensor, save_gu: bool = True,
                        ws: Optional[torch.Tensor] = None,
                        out: Optional[Dict[str, torch.Tensor]] = None):
    """Grouped SwiGLU FFN forward.  Returns dict h_perm, y_perm, gu (or None)."""
    R_cap, H = x_perm.shape
    E_l, I, _ = w_gate.shape
    dt = _dtype_code(x_perm)
    dev = x_perm.device
    o = dict(out or {})
    o.setdefault("h_perm", torch.empty((R_cap, I), dtype=x_perm.dtype, device=dev))
    o.setdefault("y_perm", torch.empty((R_cap, H), dtype=x_perm.dtype, device=dev))
    if save_gu:
        o.setdefault("gu", torch.empty((R_cap, 2 * I), dtype=x_perm.dtype, device=dev))
    else:
        o["gu"] = None
    nb = lib.moe_workspace_bytes(MOE_OP_FFN_FWD, max(R_cap, 0), H, I, max(E_l, 1), 1, 0, E_l, dt)
    if nb < 0:
        _check(int(nb), "moe_workspace_bytes")
    ws = _ws(int(nb), dev, ws)
    _check(lib.moe_grouped_ffn_fwd(_ptr(x_perm), _ptr(offsets), E_l, R_cap, H, I, _ptr(w_gate),
                                   _ptr(w_up), _ptr(w_down), dt, _ptr(o["gu"]), _ptr(o["h_perm"]),
                                   _ptr(o["y_perm"]), _ptr(ws), _nbytes(ws), _stream()),
           "moe_grouped_ffn_fwd")
    return o


def moe_grouped_ffn_fwd_gather(x: torch.Tensor, src_row: torch.Tensor, offsets: torch.Tensor,
                               w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                               R_cap: int, save_gu: bool = True, ws: Optional[torch.Tensor] = None,
                               out: Optional[Dict[str, torch.Tensor]] = None):
    """moe_grouped_ffn_fwd on the token rows x [T,H], grouped row r = x[src_row[r]]
    (moe_permute's src_row).  Returns dict h_perm, y_perm, gu (or None)."""
    T, H = x.shape
    E_l, I, _ = w_gate.shape
    dt = _dtype_code(x)
    dev = x.device
    o = dict(out or {})
    o.setdefault("h_perm", torch.empty((R_cap, I), dtype=x.dtype, device=dev))
    o.setdefault("y_perm", torch.empty((R_cap, H), dtype=x.dtype, device=dev))
    if save_gu:
        o.setdefault("gu", torch.empty((R_cap, 2 * I), dtype=x.dtype, device=dev))
    else:
        o["gu"] = None
    ws = _ws(workspace_bytes(MOE_OP_FFN_FWD, max(R_cap, 0), H, I, max(E_l, 1), 1, 0, E_l, dt), dev, ws)
    _check(lib.moe_grouped_ffn_fwd_gather(_ptr(x), _ptr(src_row), _ptr(offsets), E_l, R_cap, T, H, I,
                                          _ptr(w_gate), _ptr(w_up), _ptr(w_down), dt, _ptr(o["gu"]),
                                          _ptr(o["h_perm"]), _ptr(o["y_perm"]), _ptr(ws), _nbytes(ws),
                                          _stream()), "moe_grouped_ffn_fwd_gather")
    return o


def moe_combine(y_perm: torch.Tensor, topk_w: Optional[torch.Tensor], dest_row: torch.Tensor, T: int,
                addend: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """Weighted (or, with topk_w None, unweighted) unpermute-reduce.  Returns y [T,H]."""
    H = y_perm.shape[1]
    k = dest_row.numel() // max(T, 1)
    y = out if out is not None else torch.empty((T, H), dtype=y_perm.dtype, device=y_perm.device)
    _check(lib.moe_combine(_ptr(y_perm), _ptr(topk_w), _ptr(dest_row), _ptr(addend), T, H, k,
                           _dtype_code(y_perm), _ptr(y), _stream()), "moe_combine")
    return y


def moe_combine_bwd(dy: torch.Tensor, y_perm: torch.Tensor, topk_w: torch.Tensor,
                    dest_row: torch.Tensor, out: Optional[Dict[str, torch.Tensor]] = None):
    """Returns dict dy_perm [R_cap,H], d_topk_w [T,k]."""
    T, H = dy.shape
    k = topk_w.shape[1]
    o = dict(out or {})
    o.setdefault("dy_perm", torch.empty_like(y_perm))
    o.setdefault("d_topk_w", torch.empty((T, k), dtype=torch.float32, device=dy.device))
    _check(lib.moe_combine_bwd(_ptr(dy), _ptr(y_perm), _ptr(topk_w), _ptr(dest_row), T, H, k,
                               _dtype_code(dy), _ptr(o["dy_perm"]), _ptr(o["d_topk_w"]), _stream()),
           "moe_combine_bwd")
    return o


def moe_combine_dx(dx_perm: torch.Tensor, dest_row: torch.Tensor, d_topk_w: torch.Tensor,
                   topk_w: torch.Tensor, topk_idx: torch.Tensor, w_router: torch.Tensor,
                   ws: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """The layer's input gradient in one pass.  Returns dx [T,H] (dtype of dx_perm)."""
    T, k = topk_w.shape
    H, E = w_router.shape
    dt = _dtype_code(dx_perm)
    dx = out if out is not None else torch.empty((T, H), dtype=dx_perm.dtype, device=dx_perm.device)
    ws = _ws(workspace_bytes(MOE_OP_COMBINE_DX, T, H, 1, E, k, 0, E, dt), dx_perm.device, ws)
    _check(lib.moe_combine_dx(_ptr(dx_perm), _ptr(dest_row), _ptr(d_topk_w), _ptr(topk_w),
                              _ptr(topk_idx), _ptr(w_router), T, H, E, k, dt, _ptr(dx), _ptr(ws),
                              _nbytes(ws), _stream()), "moe_combine_dx")
    return dx


def moe_router_weight_t(w_router: torch.Tensor, out: Optional[torch.Tensor] = None):
    """The router weight [H,E] transposed to [E,H] (operand of moe_combine_dx_t)."""
    H, E = w_router.shape
    wt = out if out is not None else torch.empty((E, H), dtype=w_router.dtype, device=w_router.device)
    _check(lib.moe_router_weight_t(_ptr(w_router), H, E, _dtype_code(w_router), _ptr(wt), _stream()),
           "moe_router_weight_t")
    return wt


def moe_combine_dx_t(dx_perm: torch.Tensor, dest_row: torch.Tensor, d_topk_w: torch.Tensor,
                     topk_w: torch.Tensor, topk_idx: torch.Tensor, w_router_t: torch.Tensor,
                     out: Optional[torch.Tensor] = None):
    """moe_combine_dx with the transposed router weight [E,H].  Returns dx [T,H]."""
    T, k = topk_w.shape
    E, H = w_router_t.shape
    dx = out if out is not None else torch.empty((T, H), dtype=dx_perm.dtype, device=dx_perm.device)
    _check(lib.moe_combine_dx_t(_ptr(dx_perm), _ptr(dest_row), _ptr(d_topk_w), _ptr(topk_w),
                                _ptr(topk_idx), _ptr(w_router_t), T, H, E, k, _dtype_code(dx_perm),
                                _ptr(dx), _stream()), "moe_combine_dx_t")
    return dx


def moe_grouped_ffn_bwd(dy_perm: torch.Tensor, x_perm: torch.Tensor, gu: torch.Tensor,
                        h_perm: torch.Tensor, offsets: torch.Tensor, w_gate: torch.Tensor,
                        w_up: torch.Tensor, w_down: torch.Tensor, accumulate: bool = False,
                        ws: Optional[torch.Tensor] = None,
                        out: Optional[Dict[str, torch.Tensor]] = None):
    """Returns dict dx_perm, dw_gate, dw_up, dw_down (fp32 weight gradients)."""
    R_cap, H = x_perm.shape
    E_l, I, _ = w_gate.shape
    dt = _dtype_code(x_perm)
    dev = x_perm.device
    o = dict(out or {})
    o.setdefault("dx_perm", torch.empty_like(x_perm))
    for n, shp in (("dw_gate", (E_l, I, H)), ("dw_up", (E_l, I, H)), ("dw_down", (E_l, H, I))):
        o.setdefault(n, torch.empty(shp, dtype=torch.float32, device=dev))
    nb = lib.moe_workspace_bytes(MOE_OP_FFN_BWD, R_cap, H, I, max(E_l, 1), 1, 0, E_l, dt)
    if nb < 0:
        _check(int(nb), "moe_workspace_bytes")
    ws = _ws(int(nb), dev, ws)
    _check(lib.moe_grouped_ffn_bwd(_ptr(dy_perm), _ptr(x_perm), _ptr(gu), _ptr(h_perm),
                                   _ptr(offsets), E_l, R_cap, H, I, _ptr(w_gate), _ptr(w_up),
                                   _ptr(w_down), dt, _ptr(o["dx_perm"]), _ptr(o["dw_gate"]),
                                   _ptr(o["dw_up"]), _ptr(o["dw_down"]), int(accumulate),
                                   _ptr(ws), _nbytes(ws), _stream()), "moe_grouped_ffn_bwd")
    return o


def moe_route_bwd(d_topk_w: torch.Tensor, topk_w: torch.Tensor, topk_idx: torch.Tensor,
                  x: torch.Tensor, w_router: torch.Tensor, want_dx: bool = True,
                  want_dw: bool = True, ws: Optional[torch.Tensor] = None,
                  out: Optional[Dict[str, torch.Tensor]] = None):
    """Returns dict d_logits [T,E], dx_router [T,H] fp32 (or None), dw_router [H,E] fp32 (or None)."""
    T, H = x.shape
    E = w_router.shape[1]
    k = topk_idx.shape[1]
    dt = _dtype_code(x)
    dev = x.device
    o = dict(out or {})
    o.setdefault("d_logits", torch.empty((T, E), dtype=torch.float32, device=dev))
    if want_dx:
        o.setdefault("dx_router", torch.empty((T, H), dtype=torch.float32, device=dev))
    else:
        o["dx_router"] = None
    if want_dw:
        o.setdefault("dw_router", torch.empty((H, E), dtype=torch.float32, device=dev))
    else:
        o["dw_router"] = None
    ws = _ws(workspace_bytes(MOE_OP_ROUTE_BWD, T, H, 1, E, k, 0, E, dt), dev, ws)
    _check(lib.moe_route_bwd(_ptr(d_topk_w), _ptr(topk_w), _ptr(topk_idx), _ptr(x),
                             _ptr(w_router), T, H, E, k, dt, _ptr(o["d_logits"]),
                             _ptr(o["dx_router"]), _ptr(o["dw_router"]), _ptr(ws), _nbytes(ws),
                             _stream()), "moe_route_bwd")
    return o


# ---------------------------------------------------------------------------
# Auxiliary losses, dropout.  Their arguments are checked here for device, type
# and shape (the library sees plain pointers).  A call of a small batch takes no
# longer on the GPU than on the host, so each function first asks in one
# expression whether everything fits; where it does not (an output to allocate,
# a mistake), the checks one by one allocate or name the argument.
# ---------------------------------------------------------------------------

def _arg(t: Optional[torch.Tensor], name: str, dtype, shape, dev, optional: bool = False):
    """Pointer of a dense tensor of this type and shape on the device in use."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} must be given")
    if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    raise ValueError(f"{name} must be contiguous")


def _raw_stream(dev: torch.device) -> int:
    """The current stream of a device as a pointer (without building a Stream object, which
    costs as much as a small kernel)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _device(t: torch.Tensor) -> torch.device:
    """The device of the call: t's, which has to be the current GPU (whose current
    stream the call is enqueued on)."""
    if not t.is_cuda:
        raise ValueError(f"expected tensors on a GPU, got {t.device}")
    if t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on {t.device} while cuda:{torch.cuda.current_device()} is the "
                         f"current device")
    return t.device


def _into(o: Dict[str, torch.Tensor], name: str, shape, dtype, dev) -> int:
    """Pointer of output `name`: the caller's tensor from o (checked), else a new one."""
    if o.get(name) is None:
        o[name] = torch.empty(shape, dtype=dtype, device=dev)
        return o[name].data_ptr()
    return _arg(o[name], name, dtype, shape, dev)


@functools.lru_cache(maxsize=64)
def _balance_ws_bytes(T: int, E: int, S: int) -> int:
    nb = lib.moe_balance_ws_bytes(T, E, S)
    if nb < 0:
        _check(int(nb), "moe_balance_ws_bytes")
    return int(nb)


@functools.lru_cache(maxsize=64)
def _adapter_ws_bytes(R: int, K: int, N: int, n_ids: int, rank: int, dtype: int) -> int:
    nb = lib.moe_adapter_ws_bytes(R, K, N, n_ids, rank, dtype)
    if nb < 0:
        _check(int(nb), "moe_adapter_ws_bytes")
    return int(nb)


def _work(nbytes: int, dev, ws: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """_ws with the caller's workspace checked for the device as well."""
    if ws is not None and (ws.device != dev or not ws.is_contiguous()):
        raise ValueError(f"ws must be a contiguous tensor on {dev}, got one on {ws.device}")
    return _ws(nbytes, dev, ws)


def _int32(**sizes):
    """Refuses sizes that do not fit the library's int arguments (ctypes would cut them)."""
    for name, v in sizes.items():
        if not -(1 << 31) <= v < 1 << 31:
            raise ValueError(f"{name}={v} does not fit 32 bits")


def _row_type(t: torch.Tensor, name: str) -> torch.dtype:
    if t.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{name} must be bf16 or fp32, got {t.dtype}")
    return t.dtype


def _shape2(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, got shape {tuple(t.shape)}")
    return t.shape


def moe_route_bwd_add(d_topk_w: torch.Tensor, topk_w: torch.Tensor, topk_idx: torch.Tensor,
                      d_logits_add: torch.Tensor, x: torch.Tensor, w_router: torch.Tensor,
                      want_dx: bool = True, want_dw: bool = True, ws: Optional[torch.Tensor] = None,
                      out: Optional[Dict[str, torch.Tensor]] = None):
    """moe_route_bwd with d_logits_add [T,E] (e.g. moe_balance_loss_bwd's) added to the logit
    gradient.  Returns dict d_logits [T,E], dx_router [T,H] fp32 (or None), dw_router [H,E] fp32
    (or None); out["d_logits"] may be d_logits_add."""
    dev = _device(x)
    T, H = _shape2(x, "x")
    E = _shape2(w_router, "w_router")[1]
    k = _shape2(topk_idx, "topk_idx")[1]
    _int32(T=T, H=H, E=E, k=k)
    dt, f32 = _row_type(x, "x"), torch.float32
    o = dict(out or {})
    a = [_arg(d_topk_w, "d_topk_w", f32, (T, k), dev), _arg(topk_w, "topk_w", f32, (T, k), dev),
         _arg(topk_idx, "topk_idx", torch.int32, (T, k), dev),
         _arg(d_logits_add, "d_logits_add", f32, (T, E), dev), _arg(x, "x", dt, (T, H), dev),
         _arg(w_router, "w_router", dt, (H, E), dev)]
    d_logits = _into(o, "d_logits", (T, E), f32, dev)
    dx = _into(o, "dx_router", (T, H), f32, dev) if want_dx else None
    dw = _into(o, "dw_router", (H, E), f32, dev) if want_dw else None
    if not want_dx:
        o["dx_router"] = None
    if not want_dw:
        o["dw_router"] = None
    code = _dtype_code(x)
    ws = _work(workspace_bytes(MOE_OP_ROUTE_BWD, T, H, 1, E, k, 0, E, code), dev, ws)
    _check(lib.moe_route_bwd_add(*a, T, H, E, k, code, d_logits, dx, dw, _ptr(ws), _nbytes(ws),
                                 _raw_stream(dev)), "moe_route_bwd_add")
    return o


def _sequences(seq_offsets: Optional[torch.Tensor], dev):
    """(S, pointer): the packed sequences, or all rows as one."""
    if seq_offsets is None:
        return 1, None
    S = seq_offsets.numel() - 1
    return S, _arg(seq_offsets, "seq_offsets", torch.int32, (S + 1,), dev)


def moe_balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor, balance_coef: float,
                     z_coef: float = 0.0, seq_offsets: Optional[torch.Tensor] = None,
                     token_mask: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                     out: Optional[Dict[str, torch.Tensor]] = None):
    """Load-balance and z loss of the router's logits [T,E] fp32, with the per-expert counts.
    seq_offsets [S+1] int32: packed sequences (None: one); token_mask [T] uint8, 0 = padding.
    Returns dict loss [3] (balance, z, balance_coef * balance + z_coef * z), counts [S,E] int32,
    prob_sum [S,E], tokens [S+1] int32 (live rows of each sequence, then of all), lse [T], and the
    workspace ws used (pass it and the dict back in to allocate nothing)."""
    f32, i32, d = torch.float32, torch.int32, logits.get_device()
    o = dict(out) if out else {}
    if len(o) >= 5 and ws is not None and logits.dim() == 2 and topk_idx.dim() == 2:
        T, E = logits.shape
        k = topk_idx.shape[1]
        S = 1 if seq_offsets is None else seq_offsets.numel() - 1
        cnt, q, n, lse, loss = map(o.get, ("counts", "prob_sum", "tokens", "lse", "loss"))
        if (d >= 0 and d == torch._C._cuda_getDevice() and S > 0 and not (T | E | k | S) >> 31
                and cnt is not None and q is not None and n is not None and lse is not None
                and loss is not None
                and logits.dtype is f32 and logits.is_contiguous()
                and topk_idx.dtype is i32 and topk_idx.get_device() == d
                and topk_idx.shape[0] == T and topk_idx.is_contiguous()
                and (seq_offsets is None or seq_offsets.dtype is i32 and seq_offsets.get_device() == d
                     and seq_offsets.dim() == 1 and seq_offsets.is_contiguous())
                and (token_mask is None or token_mask.dtype is torch.uint8
                     and token_mask.get_device() == d and token_mask.shape == (T,)
                     and token_mask.is_contiguous())
                and cnt.dtype is i32 and cnt.get_device() == d and cnt.shape == (S, E)
                and cnt.is_contiguous()
                and q.dtype is f32 and q.get_device() == d and q.shape == (S, E) and q.is_contiguous()
                and n.dtype is i32 and n.get_device() == d and n.shape == (S + 1,) and n.is_contiguous()
                and lse.dtype is f32 and lse.get_device() == d and lse.shape == (T,)
                and lse.is_contiguous()
                and loss.dtype is f32 and loss.get_device() == d and loss.shape == (3,)
                and loss.is_contiguous()
                and ws.get_device() == d and ws.is_contiguous()
                and ws.nbytes >= _balance_ws_bytes(T, E, S)):
            rc = lib.moe_balance_loss(
                logits.data_ptr(), topk_idx.data_ptr(),
                None if seq_offsets is None else seq_offsets.data_ptr(),
                None if token_mask is None else token_mask.data_ptr(), T, E, k, S, balance_coef, z_coef,
                cnt.data_ptr(), q.data_ptr(), n.data_ptr(), lse.data_ptr(), loss.data_ptr(),
                ws.data_ptr(), ws.nbytes, torch._C._cuda_getCurrentRawStream(d))
            if rc != 0:
                _check(rc, "moe_balance_loss")
            o["ws"] = ws
            return o
    dev = _device(logits)
    T, E = _shape2(logits, "logits")
    k = _shape2(topk_idx, "topk_idx")[1]
    S, off = _sequences(seq_offsets, dev)
    _int32(T=T, E=E, k=k, S=S)
    a = [_arg(logits, "logits", f32, (T, E), dev), _arg(topk_idx, "topk_idx", i32, (T, k), dev), off,
         _arg(token_mask, "token_mask", torch.uint8, (T,), dev, optional=True)]
    o["ws"] = _work(_balance_ws_bytes(T, E, S), dev, ws)
    _check(lib.moe_balance_loss(*a, T, E, k, S, balance_coef, z_coef,
                                _into(o, "counts", (S, E), i32, dev),
                                _into(o, "prob_sum", (S, E), f32, dev),
                                _into(o, "tokens", (S + 1,), i32, dev), _into(o, "lse", (T,), f32, dev),
                                _into(o, "loss", (3,), f32, dev), _ptr(o["ws"]), _nbytes(o["ws"]),
                                _raw_stream(dev)), "moe_balance_loss")
    return o


def moe_balance_loss_bwd(logits: torch.Tensor, fwd: Dict[str, torch.Tensor], k: int,
                         balance_coef: float, z_coef: float = 0.0,
                         d_loss: Optional[torch.Tensor] = None,
                         seq_offsets: Optional[torch.Tensor] = None,
                         token_mask: Optional[torch.Tensor] = None, accumulate: bool = False,
                         out: Optional[torch.Tensor] = None):
    """Gradient of loss[2] wrt the logits; fwd: moe_balance_loss's dict (lse, counts, tokens) for
    the same logits, k, seq_offsets and token_mask; d_loss [1] fp32: the upstream gradient (None:
    1).  Returns d_logits [T,E] (out, added to with accumulate=True)."""
    f32, i32, d = torch.float32, torch.int32, logits.get_device()
    if out is not None and logits.dim() == 2:
        T, E = logits.shape
        S = 1 if seq_offsets is None else seq_offsets.numel() - 1
        lse, cnt, n = fwd["lse"], fwd["counts"], fwd["tokens"]
        if (d >= 0 and d == torch._C._cuda_getDevice() and S > 0 and not (T | E | k | S) >> 31
                and logits.dtype is f32 and logits.is_contiguous()
                and lse.dtype is f32 and lse.get_device() == d and lse.shape == (T,)
                and lse.is_contiguous()
                and cnt.dtype is i32 and cnt.get_device() == d and cnt.shape == (S, E)
                and cnt.is_contiguous()
                and n.dtype is i32 and n.get_device() == d and n.shape == (S + 1,) and n.is_contiguous()
                and (seq_offsets is None or seq_offsets.dtype is i32 and seq_offsets.get_device() == d
                     and seq_offsets.dim() == 1 and seq_offsets.is_contiguous())
                and (token_mask is None or token_mask.dtype is torch.uint8
                     and token_mask.get_device() == d and token_mask.shape == (T,)
                     and token_mask.is_contiguous())
                and (d_loss is None or d_loss.dtype is f32 and d_loss.get_device() == d
                     and d_loss.shape == (1,))
                and out.dtype is f32 and out.get_device() == d and out.shape == (T, E)
                and out.is_contiguous()):
            rc = lib.moe_balance_loss_bwd(
                logits.data_ptr(), lse.data_ptr(), cnt.data_ptr(), n.data_ptr(),
                None if seq_offsets is None else seq_offsets.data_ptr(),
                None if token_mask is None else token_mask.data_ptr(),
                None if d_loss is None else d_loss.data_ptr(), T, E, k, S, balance_coef, z_coef,
                1 if accumulate else 0, out.data_ptr(), torch._C._cuda_getCurrentRawStream(d))
            if rc != 0:
                _check(rc, "moe_balance_loss_bwd")
            return out
    dev = _device(logits)
    T, E = _shape2(logits, "logits")
    S, off = _sequences(seq_offsets, dev)
    _int32(T=T, E=E, k=k, S=S)
    if accumulate and out is None:
        raise ValueError("accumulate=True needs out")
    o = {"d_logits": out}
    a = [_arg(logits, "logits", f32, (T, E), dev), _arg(fwd["lse"], "lse", f32, (T,), dev),
         _arg(fwd["counts"], "counts", i32, (S, E), dev),
         _arg(fwd["tokens"], "tokens", i32, (S + 1,), dev), off,
         _arg(token_mask, "token_mask", torch.uint8, (T,), dev, optional=True),
         _arg(d_loss, "d_loss", f32, (1,), dev, optional=True)]
    _check(lib.moe_balance_loss_bwd(*a, T, E, k, S, balance_coef, z_coef, 1 if accumulate else 0,
                                    _into(o, "d_logits", (T, E), f32, dev), _raw_stream(dev)),
           "moe_balance_loss_bwd")
    return o["d_logits"]


def moe_combine_dropout(y_perm: torch.Tensor, topk_w: Optional[torch.Tensor], dest_row: torch.Tensor,
                        T: int, p: float, rng: torch.Tensor,
                        residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """moe_combine with dropout (probability p) and the residual [T,H] added.  rng [2] int64 on the
    GPU: seed and offset of the counter-based generator; the same rng goes to
    moe_combine_dropout_bwd.  Returns y [T,H] (out may be residual)."""
    dt, d = y_perm.dtype, y_perm.get_device()
    if out is not None and topk_w is not None and y_perm.dim() == 2 and topk_w.dim() == 2:
        H, k = y_perm.shape[1], topk_w.shape[1]
        if (d >= 0 and d == torch._C._cuda_getDevice() and not (T | H | k) >> 31
                and (dt is torch.bfloat16 or dt is torch.float32) and y_perm.is_contiguous()
                and topk_w.dtype is torch.float32 and topk_w.get_device() == d
                and topk_w.shape[0] == T and topk_w.is_contiguous()
                and dest_row.dtype is torch.int32 and dest_row.get_device() == d
                and dest_row.shape == (T * k,) and dest_row.is_contiguous()
                and (residual is None or residual.dtype is dt and residual.get_device() == d
                     and residual.shape == (T, H) and residual.is_contiguous())
                and rng.dtype is torch.int64 and rng.get_device() == d and rng.shape == (2,)
                and rng.is_contiguous()
                and out.dtype is dt and out.get_device() == d and out.shape == (T, H)
                and out.is_contiguous()):
            rc = lib.moe_combine_dropout(
                y_perm.data_ptr(), topk_w.data_ptr(), dest_row.data_ptr(),
                None if residual is None else residual.data_ptr(), p, rng.data_ptr(), T, H, k,
                MOE_BF16 if dt is torch.bfloat16 else MOE_F32, out.data_ptr(),
                torch._C._cuda_getCurrentRawStream(d))
            if rc != 0:
                _check(rc, "moe_combine_dropout")
            return out
    dev = _device(y_perm)
    R_cap, H = _shape2(y_perm, "y_perm")
    dt = _row_type(y_perm, "y_perm")
    if T < 0 or dest_row.numel() % max(T, 1):
        raise ValueError(f"dest_row has {dest_row.numel()} entries, not a multiple of T = {T}")
    k = topk_w.shape[1] if topk_w is not None and topk_w.dim() == 2 else dest_row.numel() // max(T, 1) or 1
    _int32(T=T, H=H, k=k)
    if out is None:
        out = torch.empty((T, H), dtype=dt, device=dev)
    rc = lib.moe_combine_dropout(
        _arg(y_perm, "y_perm", dt, (R_cap, H), dev),
        None if topk_w is None else _arg(topk_w, "topk_w", torch.float32, (T, k), dev),
        _arg(dest_row, "dest_row", torch.int32, (T * k,), dev),
        None if residual is None else _arg(residual, "residual", dt, (T, H), dev), p,
        _arg(rng, "rng", torch.int64, (2,), dev), T, H, k,
        MOE_BF16 if dt is torch.bfloat16 else MOE_F32, _arg(out, "out", dt, (T, H), dev), _raw_stream(dev))
    if rc != 0:
        _check(rc, "moe_combine_dropout")
    return out


def moe_combine_dropout_bwd(dy: torch.Tensor, y_perm: torch.Tensor, topk_w: torch.Tensor,
                            dest_row: torch.Tensor, p: float, rng: torch.Tensor,
                            out: Optional[Dict[str, torch.Tensor]] = None):
    """Backward of moe_combine_dropout under its p and rng (the residual's gradient is dy).
    Returns dict dy_perm [R_cap,H], d_topk_w [T,k]."""
    dt, f32, d = dy.dtype, torch.float32, dy.get_device()
    o = dict(out) if out else {}
    dyp, dw = o.get("dy_perm"), o.get("d_topk_w")
    if (dyp is not None and dw is not None and dy.dim() == 2 and topk_w.dim() == 2
            and y_perm.dim() == 2):
        T, H = dy.shape
        k = topk_w.shape[1]
        if (d >= 0 and d == torch._C._cuda_getDevice() and not (T | H | k) >> 31
                and (dt is torch.bfloat16 or dt is torch.float32) and dy.is_contiguous()
                and y_perm.dtype is dt and y_perm.get_device() == d and y_perm.shape[1] == H
                and y_perm.is_contiguous()
                and topk_w.dtype is f32 and topk_w.get_device() == d and topk_w.shape[0] == T
                and topk_w.is_contiguous()
                and dest_row.dtype is torch.int32 and dest_row.get_device() == d
                and dest_row.shape == (T * k,) and dest_row.is_contiguous()
                and rng.dtype is torch.int64 and rng.get_device() == d and rng.shape == (2,)
                and rng.is_contiguous()
                and dyp.dtype is dt and dyp.get_device() == d and dyp.shape == y_perm.shape
                and dyp.is_contiguous()
                and dw.dtype is f32 and dw.get_device() == d and dw.shape == (T, k)
                and dw.is_contiguous()):
            rc = lib.moe_combine_dropout_bwd(
                dy.data_ptr(), y_perm.data_ptr(), topk_w.data_ptr(), dest_row.data_ptr(), p,
                rng.data_ptr(), T, H, k, MOE_BF16 if dt is torch.bfloat16 else MOE_F32,
                dyp.data_ptr(), dw.data_ptr(), torch._C._cuda_getCurrentRawStream(d))
            if rc != 0:
                _check(rc, "moe_combine_dropout_bwd")
            return o
    dev = _device(dy)
    T, H = _shape2(dy, "dy")
    k = _shape2(topk_w, "topk_w")[1]
    R_cap = _shape2(y_perm, "y_perm")[0]
    _int32(T=T, H=H, k=k)
    dt = _row_type(dy, "dy")
    a = [_arg(dy, "dy", dt, (T, H), dev), _arg(y_perm, "y_perm", dt, (R_cap, H), dev),
         _arg(topk_w, "topk_w", f32, (T, k), dev),
         _arg(dest_row, "dest_row", torch.int32, (T * k,), dev)]
    _check(lib.moe_combine_dropout_bwd(*a, p, _arg(rng, "rng", torch.int64, (2,), dev), T, H, k,
                                       _dtype_code(dy), _into(o, "dy_perm", (R_cap, H), dt, dev),
                                       _into(o, "d_topk_w", (T, k), f32, dev), _raw_stream(dev)),
           "moe_combine_dropout_bwd")
    return o


def _rows_arg(t: torch.Tensor, name: str, dtype, rows: int, cols: int, dev):
    """(pointer, row pitch) of a matrix whose rows are dense, at any pitch."""
    if t.dtype is dtype and t.shape == (rows, cols) and t.device == dev and t.is_contiguous():
        return t.data_ptr(), cols
    if t.dtype != dtype or t.shape != (rows, cols) or t.device != dev:
        raise ValueError(f"{name} must be {dtype} [{rows}, {cols}] on {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    ld = t.stride(0) if rows > 1 else cols
    if (cols > 1 and t.stride(1) != 1) or ld < cols:
        raise ValueError(f"{name} must have dense rows that do not overlap, got strides {t.stride()}")
    _int32(**{f"the row pitch of {name}": ld})
    return t.data_ptr(), ld


def _adapter_args(x, row_id, A, B, scale, src_row):
    """Checked arguments that moe_adapter_fwd and _bwd share."""
    dev = _device(row_id)
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("A must be [n_ids, rank, K] and B [n_ids, N, rank]")
    n_ids, rank, K = A.shape
    N, R = B.shape[1], row_id.numel()
    dt, i32 = _row_type(A, "A"), torch.int32
    x_rows = _shape2(x, "x")[0]
    _int32(R=R, x_rows=x_rows, K=K, N=N, n_ids=n_ids, rank=rank)
    if src_row is None and x_rows != R:
        raise ValueError(f"x has {x_rows} rows, row_id {R} (src_row maps one to the other)")
    ptrs = (_arg(src_row, "src_row", i32, (R,), dev, optional=True), _arg(row_id, "row_id", i32, (R,), dev),
            _arg(A, "A", dt, (n_ids, rank, K), dev), _arg(B, "B", dt, (n_ids, N, rank), dev))
    sc = _arg(scale, "scale", torch.float32, (n_ids,), dev, optional=True)
    xp, ldx = _rows_arg(x, "x", dt, x_rows, K, dev)
    return dev, dt, n_ids, rank, K, N, R, x_rows, xp, ldx, ptrs, sc


def moe_adapter_fwd(x: torch.Tensor, row_id: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                    y: torch.Tensor, scale: Optional[torch.Tensor] = None,
                    src_row: Optional[torch.Tensor] = None, want_v: bool = False,
                    out: Optional[torch.Tensor] = None):
    """Low-rank adapters added to y [R,N] in place: row r gets
    scale[a] * B[a] (A[a] x[src_row[r]]), a = row_id[r] (-1: none).  A [n_ids,rank,K],
    B [n_ids,N,rank]; rows of x and y may lie at any pitch.  Returns v [R,rank] fp32 for
    moe_adapter_bwd with want_v=True (written to out if given), else None."""
    d, dt, i32 = row_id.get_device(), A.dtype, torch.int32
    if A.dim() == 3 and B.dim() == 3 and x.dim() == 2 and (not want_v or out is not None):
        n_ids, rank, K = A.shape
        N, R, x_rows = B.shape[1], row_id.numel(), x.shape[0]
        if (d >= 0 and d == torch._C._cuda_getDevice() and not (R | x_rows | K | N | n_ids | rank) >> 31
                and (dt is torch.bfloat16 or dt is torch.float32)
                and A.get_device() == d and A.is_contiguous()
                and B.dtype is dt and B.get_device() == d and B.shape == (n_ids, N, rank)
                and B.is_contiguous()
                and row_id.dtype is i32 and row_id.dim() == 1 and row_id.is_contiguous()
                and x.dtype is dt and x.get_device() == d and x.shape[1] == K and x.is_contiguous()
                and y.dtype is dt and y.get_device() == d and y.shape == (R, N) and y.is_contiguous()
                and (scale is None or scale.dtype is torch.float32 and scale.get_device() == d
                     and scale.shape == (n_ids,) and scale.is_contiguous())
                and (x_rows == R if src_row is None else
                     src_row.dtype is i32 and src_row.get_device() == d
                     and src_row.shape == (R,) and src_row.is_contiguous())
                and (not want_v or out.dtype is torch.float32 and out.get_device() == d
                     and out.shape == (R, rank) and out.is_contiguous())):
            rc = lib.moe_adapter_fwd(
                x.data_ptr(), None if src_row is None else src_row.data_ptr(), row_id.data_ptr(),
                A.data_ptr(), B.data_ptr(), None if scale is None else scale.data_ptr(), R, x_rows, K, N,
                K, N, n_ids, rank, MOE_BF16 if dt is torch.bfloat16 else MOE_F32, y.data_ptr(),
                out.data_ptr() if want_v else None, torch._C._cuda_getCurrentRawStream(d))
            if rc != 0:
                _check(rc, "moe_adapter_fwd")
            return out if want_v else None
    dev, dt, n_ids, rank, K, N, R, x_rows, xp, ldx, (src, ids, a, b), sc = \
        _adapter_args(x, row_id, A, B, scale, src_row)
    yp, ldy = _rows_arg(y, "y", dt, R, N, dev)
    v = None
    if want_v:
        if out is None:
            out = torch.empty((R, rank), dtype=torch.float32, device=dev)
        v = _arg(out, "out", torch.float32, (R, rank), dev)
    rc = lib.moe_adapter_fwd(xp, src, ids, a, b, sc, R, x_rows, K, N, ldx, ldy, n_ids, rank,
                             MOE_BF16 if dt is torch.bfloat16 else MOE_F32, yp, v, _raw_stream(dev))
    if rc != 0:
        _check(rc, "moe_adapter_fwd")
    return out if want_v else None


def moe_adapter_bwd(dy: torch.Tensor, x: torch.Tensor, row_id: torch.Tensor, A: torch.Tensor,
                    B: torch.Tensor, v: Optional[torch.Tensor], dx: Optional[torch.Tensor],
                    scale: Optional[torch.Tensor] = None, src_row: Optional[torch.Tensor] = None,
                    want_dw: bool = True, accumulate: bool = False,
                    ws: Optional[torch.Tensor] = None,
                    out: Optional[Dict[str, torch.Tensor]] = None):
    """Backward of moe_adapter_fwd for dy [R,N] and the forward's v: dx [R,K] (None: not wanted)
    is added to in place.  Returns dict dA [n_ids,rank,K], dB [n_ids,N,rank] fp32 (None with
    want_dw=False; added to with accumulate=True) and the workspace ws used."""
    d, dt, i32, f32 = row_id.get_device(), A.dtype, torch.int32, torch.float32
    o = dict(out) if out else {}
    dA, dB = o.get("dA"), o.get("dB")
    if (dA is not None and dB is not None and want_dw and ws is not None and v is not None
            and A.dim() == 3 and B.dim() == 3 and x.dim() == 2):
        n_ids, rank, K = A.shape
        N, R, x_rows = B.shape[1], row_id.numel(), x.shape[0]
        code = MOE_BF16 if dt is torch.bfloat16 else MOE_F32
        if (d >= 0 and d == torch._C._cuda_getDevice() and not (R | x_rows | K | N | n_ids | rank) >> 31
                and (dt is torch.bfloat16 or dt is torch.float32)
                and A.get_device() == d and A.is_contiguous()
                and B.dtype is dt and B.get_device() == d and B.shape == (n_ids, N, rank)
                and B.is_contiguous()
                and row_id.dtype is i32 and row_id.dim() == 1 and row_id.is_contiguous()
                and x.dtype is dt and x.get_device() == d and x.shape[1] == K and x.is_contiguous()
                and dy.dtype is dt and dy.get_device() == d and dy.shape == (R, N) and dy.is_contiguous()
                and (dx is None or dx.dtype is dt and dx.get_device() == d and dx.shape == (R, K)
                     and dx.is_contiguous())
                and v.dtype is f32 and v.get_device() == d and v.shape == (R, rank) and v.is_contiguous()
                and dA.dtype is f32 and dA.get_device() == d and dA.shape == A.shape
                and dA.is_contiguous()
                and dB.dtype is f32 and dB.get_device() == d and dB.shape == B.shape
                and dB.is_contiguous()
                and (scale is None or scale.dtype is f32 and scale.get_device() == d
                     and scale.shape == (n_ids,) and scale.is_contiguous())
                and (x_rows == R if src_row is None else
                     src_row.dtype is i32 and src_row.get_device() == d
                     and src_row.shape == (R,) and src_row.is_contiguous())
                and ws.get_device() == d and ws.is_contiguous()
                and ws.nbytes >= _adapter_ws_bytes(R, K, N, n_ids, rank, code)):
            rc = lib.moe_adapter_bwd(
                dy.data_ptr(), x.data_ptr(), None if src_row is None else src_row.data_ptr(),
                row_id.data_ptr(), A.data_ptr(), B.data_ptr(), v.data_ptr(),
                None if scale is None else scale.data_ptr(), R, x_rows, K, N, K, N, K, n_ids, rank, code,
                None if dx is None else dx.data_ptr(), dA.data_ptr(), dB.data_ptr(),
                1 if accumulate else 0, ws.data_ptr(), ws.nbytes,
                torch._C._cuda_getCurrentRawStream(d))
            if rc != 0:
                _check(rc, "moe_adapter_bwd")
            o["ws"] = ws
            return o
    dev, dt, n_ids, rank, K, N, R, x_rows, xp, ldx, (src, ids, a, b), sc = \
        _adapter_args(x, row_id, A, B, scale, src_row)
    dyp, ldy = _rows_arg(dy, "dy", dt, R, N, dev)
    dxp, lddx = _rows_arg(dx, "dx", dt, R, K, dev) if dx is not None else (None, K)
    if accumulate and want_dw and (o.get("dA") is None or o.get("dB") is None):
        raise ValueError("accumulate=True needs out with dA and dB")
    dA = _into(o, "dA", (n_ids, rank, K), f32, dev) if want_dw else None
    dB = _into(o, "dB", (n_ids, N, rank), f32, dev) if want_dw else None
    if not want_dw:
        o["dA"] = o["dB"] = None
    vp = _arg(v, "v", f32, (R, rank), dev, optional=not want_dw)
    o["ws"] = _work(_adapter_ws_bytes(R, K, N, n_ids, rank, _dtype_code(A)), dev, ws)
    _check(lib.moe_adapter_bwd(dyp, xp, src, ids, a, b, vp, sc, R, x_rows, K, N, ldx, ldy, lddx,
                               n_ids, rank, _dtype_code(A), dxp, dA, dB, 1 if accumulate else 0,
                               _ptr(o["ws"]), _nbytes(o["ws"]), _raw_stream(dev)), "moe_adapter_bwd")
    return o


def moe_adapter_rows(offsets: torch.Tensor, src_row: torch.Tensor, token_adapter: torch.Tensor,
                     n_adapters: int, out: Optional[torch.Tensor] = None):
    """Adapter ids of moe_permute's grouped rows for adapters held per expert: row_id [R_cap] =
    token_adapter[src_row[r]] * E_l + expert of r, or -1."""
    dev = _device(offsets)
    E_l, R_cap, T = offsets.numel() - 1, src_row.numel(), token_adapter.numel()
    _int32(E_l=E_l, R_cap=R_cap, T=T, n_adapters=n_adapters)
    i32 = torch.int32
    o = {"row_id": out}
    _check(lib.moe_adapter_rows(_arg(offsets, "offsets", i32, (E_l + 1,), dev),
                                _arg(src_row, "src_row", i32, (R_cap,), dev),
                                _arg(token_adapter, "token_adapter", i32, (T,), dev), E_l, T,
                                n_adapters, R_cap, _into(o, "row_id", (R_cap,), i32, dev), _raw_stream(dev)),
           "moe_adapter_rows")
    return o["row_id"]


def moe_grouped_ffn_fwd_adapter(x: torch.Tensor, src_row: Optional[torch.Tensor],
                                offsets: torch.Tensor, row_id: torch.Tensor, w_gate: torch.Tensor,
                                w_up: torch.Tensor, w_down: torch.Tensor,
                                adapters: Dict[str, tuple], scale: Optional[torch.Tensor] = None,
                                ws: Optional[torch.Tensor] = None,
                                out: Optional[Dict[str, torch.Tensor]] = None):
    """Grouped SwiGLU FFN forward with low-rank adapters on the expert projections.  x: the
    grouped rows (src_row None) or, bf16, the token rows with moe_permute's src_row; row_id from
    moe_adapter_rows; adapters: {"gate"|"up"|"down": (A, B)}, A [n_ids, rank, in] and B [n_ids,
    out, rank] of one n_ids and rank (None: as if not given).  Returns dict h_perm, y_perm, gu."""
    dev = _device(x)
    dt = _row_type(x, "x")
    x_rows, H = _shape2(x, "x")
    E_l, I = w_gate.shape[:2]
    R_cap = row_id.numel()
    i32 = torch.int32
    unknown = set(adapters) - {"gate", "up", "down"}
    adapters = {name: pair for name, pair in adapters.items() if pair is not None}
    if unknown or not adapters:
        raise ValueError(f"adapters must name some of gate, up, down, got "
                         f"{sorted(unknown.union(adapters))}")
    n_ids, rank = next(iter(adapters.values()))[0].shape[:2]
    _int32(E_l=E_l, R_cap=R_cap, x_rows=x_rows, H=H, I=I, n_ids=n_ids, rank=rank)
    ab = []
    for name, k, n in (("gate", H, I), ("up", H, I), ("down", I, H)):
        pair = adapters.get(name)
        ab += [None, None] if pair is None else [
            _arg(pair[0], f"A of {name}", dt, (n_ids, rank, k), dev),
            _arg(pair[1], f"B of {name}", dt, (n_ids, n, rank), dev)]
    a = [_arg(x, "x", dt, (x_rows, H), dev), _arg(src_row, "src_row", i32, (R_cap,), dev, optional=True),
         _arg(offsets, "offsets", i32, (E_l + 1,), dev), _arg(row_id, "row_id", i32, (R_cap,), dev)]
    w = [_arg(w_gate, "w_gate", dt, (E_l, I, H), dev), _arg(w_up, "w_up", dt, (E_l, I, H), dev),
         _arg(w_down, "w_down", dt, (E_l, H, I), dev)]
    o = dict(out or {})
    code = _dtype_code(x)
    ws = _work(workspace_bytes(MOE_OP_FFN_FWD, R_cap, H, I, E_l, 1, 0, E_l, code), dev, ws)
    _check(lib.moe_grouped_ffn_fwd_adapter(
        *a, E_l, R_cap, x_rows, H, I, *w, *ab,
        _arg(scale, "scale", torch.float32, (n_ids,), dev, optional=True), n_ids, rank, code,
        _into(o, "gu", (R_cap, 2 * I), dt, dev), _into(o, "h_perm", (R_cap, I), dt, dev),
        _into(o, "y_perm", (R_cap, H), dt, dev), _ptr(ws), _nbytes(ws), _raw_stream(dev)),
        "moe_grouped_ffn_fwd_adapter")
    return o


from .layer import MoELayer  # noqa: E402,F401


def moe_quantize_fp8(src: torch.Tensor, nrows: Optional[torch.Tensor] = None,
                     out: Optional[Dict[str, torch.Tensor]] = None):
    """E4M3 codes of the rows of src [rows, cols] (bf16 / fp32), one power-of-two scale
    per row.  nrows: optional int32 device tensor whose first element bounds the
    rows written.  Returns (q uint8 [rows, cols], scale fp32 [rows])."""
    rows, cols = src.shape
    o = dict(out or {})
    o.setdefault("q", torch.empty((rows, cols), dtype=torch.uint8, device=src.device))
    o.setdefault("scale", torch.empty(rows, dtype=torch.float32, device=src.device))
    _check(lib.moe_quantize_fp8(_ptr(src), rows, cols, _dtype_code(src), _ptr(nrows), _ptr(o["q"]),
                                _ptr(o["scale"]), _stream()), "moe_quantize_fp8")
    return o["q"], o["scale"]


def moe_grouped_ffn_fwd_fp8(x_q: torch.Tensor, x_scale: torch.Tensor, src_row: torch.Tensor,
                            offsets: torch.Tensor, wg: tuple, wu: tuple, wd: tuple,
                            save_gu: bool = False, ws: Optional[torch.Tensor] = None,
                            out: Optional[Dict[str, torch.Tensor]] = None, R_cap: Optional[int] = None):
    """Grouped SwiGLU FFN forward on E4M3 codes.  x_q [R_cap, H] uint8 (permuted
    rows), x_scale [T] per-token scales, src_row [R_cap]; wg / wu / wd = (codes
    uint8 [E_l, N, K], scales fp32 [E_l, N]).  Returns dict h_perm, y_perm (bf16)
    and gu (or None).  With R_cap given, x_q is the token code rows [T, H] read
    through src_row (moe_grouped_ffn_fwd_fp8_gather)."""
    gather = R_cap is not None
    T, H = x_q.shape
    R_cap = R_cap if gather else T
    E_l, I, _ = wg[0].shape
    dev = x_q.device
    o = dict(out or {})
    o.setdefault("h_perm", torch.empty((R_cap, I), dtype=torch.bfloat16, device=dev))
    o.setdefault("y_perm", torch.empty((R_cap, H), dtype=torch.bfloat16, device=dev))
    if save_gu:
        o.setdefault("gu", torch.empty((R_cap, 2 * I), dtype=torch.bfloat16, device=dev))
    else:
        o["gu"] = None
    nb = lib.moe_workspace_bytes(MOE_OP_FFN_FWD_FP8, max(R_cap, 0), H, I, max(E_l, 1), 1, 0, E_l,
                                 MOE_BF16)
    if nb < 0:
        _check(int(nb), "moe_workspace_bytes")
    ws = _ws(int(nb), dev, ws)
    if gather:
        _check(lib.moe_grouped_ffn_fwd_fp8_gather(
            _ptr(x_q), _ptr(x_scale), _ptr(src_row), _ptr(offsets), E_l, R_cap, T, H, I, _ptr(wg[0]),
            _ptr(wg[1]), _ptr(wu[0]), _ptr(wu[1]), _ptr(wd[0]), _ptr(wd[1]), _ptr(o["gu"]),
            _ptr(o["h_perm"]), _ptr(o["y_perm"]), _ptr(ws), _nbytes(ws), _stream()),
            "moe_grouped_ffn_fwd_fp8_gather")
        return o
    _check(lib.moe_grouped_ffn_fwd_fp8(_ptr(x_q), _ptr(x_scale), _ptr(src_row), _ptr(offsets), E_l,
                                       R_cap, H, I, _ptr(wg[0]), _ptr(wg[1]), _ptr(wu[0]),
                                       _ptr(wu[1]), _ptr(wd[0]), _ptr(wd[1]), _ptr(o["gu"]),
                                       _ptr(o["h_perm"]), _ptr(o["y_perm"]), _ptr(ws), _nbytes(ws),
                                       _stream()), "moe_grouped_ffn_fwd_fp8")
    return o


def moe_quantize_fp8_t(w0: torch.Tensor, w1: Optional[torch.Tensor] = None,
                       out: Optional[Dict[str, torch.Tensor]] = None):
    """Per-input-channel E4M3 codes of bf16 expert weights w0 (and w1) [E_l, N, K]:
    rows of [w0^T | w1^T].  Returns (q uint8 [E_l, K, n N], scale fp32 [E_l, K])."""
    B, N, K = w0.shape
    n = 1 if w1 is None else 2
    o = dict(out or {})
    o.setdefault("q", torch.empty((B, K, n * N), dtype=torch.uint8, device=w0.device))
    o.setdefault("scale", torch.empty((B, K), dtype=torch.float32, device=w0.device))
    _check(lib.moe_quantize_fp8_t(_ptr(w0), _ptr(w1), B, N, K, _dtype_code(w0), _ptr(o["q"]),
                                  _ptr(o["scale"]), _stream()), "moe_quantize_fp8_t")
    return o["q"], o["scale"]


def moe_grouped_ffn_dgrad_fp8(dy_q: torch.Tensor, dy_scale: torch.Tensor, gu: torch.Tensor,
                              offsets: torch.Tensor, wdt: tuple, wgut: tuple,
                              ws: Optional[torch.Tensor] = None,
                              out: Optional[Dict[str, torch.Tensor]] = None):
    """Data gradients of the grouped SwiGLU FFN on E4M3 codes.  dy_q [R_cap, H] uint8
    with per-row dy_scale [R_cap]; gu [R_cap, 2I] bf16 (saved g, u); wdt = (codes
    [E_l, I, H], scales [E_l, I]) of W_down^T; wgut = (codes [E_l, H, 2I], scales
    [E_l, H]) of [W_gate^T | W_up^T].  Returns dict dgu [R_cap, 2I] and dx_perm
    [R_cap, H] (bf16)."""
    R_cap, H = dy_q.shape
    E_l, I, _ = wdt[0].shape
    dev = dy_q.device
    o = dict(out or {})
    o.setdefault("dgu", torch.empty((R_cap, 2 * I), dtype=torch.bfloat16, device=dev))
    o.setdefault("dx_perm", torch.empty((R_cap, H), dtype=torch.bfloat16, device=dev))
    nb = lib.moe_workspace_bytes(MOE_OP_FFN_DGRAD_FP8, max(R_cap, 0), H, I, max(E_l, 1), 1, 0, E_l,
                                 MOE_BF16)
    if nb < 0:
        _check(int(nb), "moe_workspace_bytes")
    ws = _ws(int(nb), dev, ws)
    _check(lib.moe_grouped_ffn_dgrad_fp8(_ptr(dy_q), _ptr(dy_scale), _ptr(gu), _ptr(offsets), E_l,
                                         R_cap, H, I, _ptr(wdt[0]), _ptr(wdt[1]), _ptr(wgut[0]),
                                         _ptr(wgut[1]), _ptr(o["dgu"]), _ptr(o["dx_perm"]),
                                         _ptr(ws), _nbytes(ws), _stream()),
           "moe_grouped_ffn_dgrad_fp8")
    return o


def wgrad_fp8_pitch(R_cap: int, E_l: int) -> int:
    """Row pitch (codes) of the transposed code matrices: room for every group's
    rows rounded up to 64."""
    return ((R_cap + 63) // 64) * 64 + 64 * E_l


def moe_quantize_fp8_group_t(src: torch.Tensor, offsets: torch.Tensor, E_l: int,
                             src_row: Optional[torch.Tensor] = None, R_cap: Optional[int] = None,
                             out: Optional[Dict[str, torch.Tensor]] = None):
    """Per-(group, column) E4M3 codes of grouped bf16 rows (row r = src[src_row[r]] if
    src_row is given, else src[r]), transposed: returns dict q uint8 [C, pitch]
    (group g at columns poff[g] ..), scale fp32 [E_l, C], poff int32 [E_l + 1]."""
    C = src.shape[1]
    if R_cap is None:
        R_cap = src_row.numel() if src_row is not None else src.shape[0]
    pitch = wgrad_fp8_pitch(R_cap, E_l)
    dev = src.device
    o = dict(out or {})
    o.setdefault("q", torch.empty((C, pitch), dtype=torch.uint8, device=dev))
    o.setdefault("scale", torch.empty((E_l, C), dtype=torch.float32, device=dev))
    o.setdefault("poff", torch.empty(E_l + 1, dtype=torch.int32, device=dev))
    _check(lib.moe_quantize_fp8_group_t(_ptr(src), _ptr(src_row), C, _ptr(offsets), E_l, R_cap,
                                        _ptr(o["q"]), o["q"].shape[1], _ptr(o["scale"]),
                                        _ptr(o["poff"]), _stream()), "moe_quantize_fp8_group_t")
    return o


def moe_grouped_ffn_wgrad_fp8(x: torch.Tensor, src_row: Optional[torch.Tensor], dgu: torch.Tensor,
                              h_perm: torch.Tensor, dy_perm: torch.Tensor, offsets: torch.Tensor,
                              E_l: int, accumulate: bool = False, ws: Optional[torch.Tensor] = None,
                              out: Optional[Dict[str, torch.Tensor]] = None):
    """Weight gradients of the grouped SwiGLU FFN on E4M3 codes (operands quantized per
    (expert, column)).  x [T, H] with src_row [R_cap] (or the grouped rows [R_cap, H]
    with src_row None), dgu [R_cap, 2I], h_perm [R_cap, I], dy_perm [R_cap, H], all
    bf16.  Returns dict dw_gate, dw_up [E_l, I, H] and dw_down [E_l, H, I] (fp32)."""
    R_cap, H = dy_perm.shape
    I = h_perm.shape[1]
    dev = dy_perm.device
    o = dict(out or {})
    for n, sh in (("dw_gate", (E_l, I, H)), ("dw_up", (E_l, I, H)), ("dw_down", (E_l, H, I))):
        o.setdefault(n, torch.empty(sh, dtype=torch.float32, device=dev))
    nb = lib.moe_workspace_bytes(MOE_OP_FFN_WGRAD_FP8, max(R_cap, 0), H, I, max(E_l, 1), 1, 0, E_l,
                                 MOE_BF16)
    if nb < 0:
        _check(int(nb), "moe_workspace_bytes")
    ws = _ws(int(nb), dev, ws)
    _check(lib.moe_grouped_ffn_wgrad_fp8(_ptr(x), _ptr(src_row), _ptr(dgu), _ptr(h_perm),
                                         _ptr(dy_perm), _ptr(offsets), E_l, R_cap, H, I,
                                         _ptr(o["dw_gate"]), _ptr(o["dw_up"]), _ptr(o["dw_down"]),
                                         1 if accumulate else 0, _ptr(ws), _nbytes(ws), _stream()),
           "moe_grouped_ffn_wgrad_fp8")
    return o


def _wgrad_fp8_ws(R_cap, H, I, E_l, dev, ws):
    nb = lib.moe_workspace_bytes(MOE_OP_FFN_WGRAD_FP8, max(R_cap, 0), H, I, max(E_l, 1), 1, 0, E_l,
                                 MOE_BF16)
    if nb < 0:
        _check(int(nb), "moe_workspace_bytes")
    return _ws(int(nb), dev, ws)


def moe_grouped_ffn_wgrad_fp8_begin(x: torch.Tensor, src_row: Optional[torch.Tensor],
                                    h_perm: torch.Tensor, dy_perm: torch.Tensor,
                                    offsets: torch.Tensor, E_l: int, ws: torch.Tensor,
                                    dw_down: torch.Tensor, accumulate: bool = False, stream=None):
    """First half of moe_grouped_ffn_wgrad_fp8: the columns of x (through src_row),
    dy_perm and h_perm quantized into ws, the K-chunk plans, dW_down (complete only
    after moe_grouped_ffn_wgrad_fp8_end on the same ws).  stream: a torch stream
    (default: the current one)."""
    R_cap, H = dy_perm.shape
    I = h_perm.shape[1]
    ws = _wgrad_fp8_ws(R_cap, H, I, E_l, dy_perm.device, ws)
    st = (stream or torch.cuda.current_stream()).cuda_stream
    _check(lib.moe_grouped_ffn_wgrad_fp8_begin(_ptr(x), _ptr(src_row), _ptr(h_perm), _ptr(dy_perm),
                                               _ptr(offsets), E_l, R_cap, H, I, _ptr(dw_down),
                                               1 if accumulate else 0, _ptr(ws), _nbytes(ws),
                                               ctypes.c_void_p(st)),
           "moe_grouped_ffn_wgrad_fp8_begin")


def moe_grouped_ffn_wgrad_fp8_end(dgu: torch.Tensor, offsets: torch.Tensor, E_l: int, H: int,
                                  ws: torch.Tensor, out: Dict[str, torch.Tensor],
                                  accumulate: bool = False, stream=None):
    """Second half: the columns of dgu [R_cap, 2I] quantized, dW_gate and dW_up, and
    the split experts' partial sums of both products (out: dw_gate, dw_up, and the
    dw_down that begin wrote)."""
    R_cap, I2 = dgu.shape
    I = I2 // 2
    ws = _wgrad_fp8_ws(R_cap, H, I, E_l, dgu.device, ws)
    st = (stream or torch.cuda.current_stream()).cuda_stream
    _check(lib.moe_grouped_ffn_wgrad_fp8_end(_ptr(dgu), _ptr(offsets), E_l, R_cap, H, I,
                                             _ptr(out["dw_gate"]), _ptr(out["dw_up"]),
                                             _ptr(out["dw_down"]), 1 if accumulate else 0, _ptr(ws),
                                             _nbytes(ws), ctypes.c_void_p(st)),
           "moe_grouped_ffn_wgrad_fp8_end")


def moe_quantize_fp8_w(w0: torch.Tensor, w1: Optional[torch.Tensor] = None, transposed: bool = True,
                       ws: Optional[torch.Tensor] = None,
                       out: Optional[Dict[str, torch.Tensor]] = None):
    """Both E4M3 code layouts of bf16 expert weights w0 (and w1) [B, N, K]: the rows
    (q0/s0, q1/s1, as moe_quantize_fp8) and, unless transposed is False, the rows of
    [w0^T | w1^T] (qt [B, K, n N] / st [B, K], as moe_quantize_fp8_t)."""
    B, N, K = w0.shape
    n = 1 if w1 is None else 2
    dev = w0.device
    o = dict(out or {})
    o.setdefault("q0", torch.empty((B, N, K), dtype=torch.uint8, device=dev))
    o.setdefault("s0", torch.empty((B, N), dtype=torch.float32, device=dev))
    if w1 is not None:
        o.setdefault("q1", torch.empty((B, N, K), dtype=torch.uint8, device=dev))
        o.setdefault("s1", torch.empty((B, N), dtype=torch.float32, device=dev))
    else:
        o["q1"] = o["s1"] = None
    if transposed:
        o.setdefault("qt", torch.empty((B, K, n * N), dtype=torch.uint8, device=dev))
        o.setdefault("st", torch.empty((B, K), dtype=torch.float32, device=dev))
    else:
        o["qt"] = o["st"] = None
    al = lambda b: (b + 255) // 256 * 256
    nb = 2 * al(n * B * N * (K // 128) * 4) + al(n * B * N * 4) + al(B * K * 4)
    ws = _ws(nb, dev, ws)
    _check(lib.moe_quantize_fp8_w(_ptr(w0), _ptr(w1), B, N, K, _dtype_code(w0), _ptr(o["q0"]),
                                  _ptr(o["s0"]), _ptr(o["q1"]), _ptr(o["s1"]), _ptr(o["qt"]),
                                  _ptr(o["st"]), _ptr(ws), _nbytes(ws), _stream()),
           "moe_quantize_fp8_w")
    return o
