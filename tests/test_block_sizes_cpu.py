"""Sizes that do not fit the library's int32 arguments are refused by the binding of the norms and of the
8-bit rows and products, not cut to their low bits (tensors without memory stand in for those on a GPU)."""
import pytest
import torch

import moe_expert_layer_router_amd as moe
from moe_expert_layer_router_amd import int8, norm

BIG = (1 << 32) + 16  # 16 in its low 32 bits
bf, f32, i32, i8 = torch.bfloat16, torch.float32, torch.int32, torch.int8


def t(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="meta")


W = (t(i8, 2, 32, 64), t(f32, 2, 32))
CALLS = {
    "moe_norm": lambda n: moe.moe_norm(t(bf, n, 8), t(f32, 8)),
    "moe_norm width": lambda n: moe.moe_norm(t(bf, 4, n), t(f32, n)),
    "moe_norm_bwd": lambda n: moe.moe_norm_bwd(t(bf, n, 8), t(bf, n, 8), t(f32, 8)),
    "moe_combine_norm": lambda n: moe.moe_combine_norm(t(bf, 6, 8), None, t(i32, n), n, t(f32, 8)),
    "moe_combine_norm_bwd": lambda n: moe.moe_combine_norm_bwd(t(bf, n, 8), t(bf, 6, 8), t(f32, n, 1), t(i32, n),
                                                               t(f32, 8)),
    "moe_quantize_i8": lambda n: moe.moe_quantize_i8(t(bf, n, 16)),
    "moe_quantize_i8 3d": lambda n: moe.moe_quantize_i8(t(bf, n // 16, 16, 16)),
    "moe_dequantize_i8": lambda n: moe.moe_dequantize_i8(t(i8, n, 16), t(f32, n), bf),
    "moe_dequantize_i8 map": lambda n: moe.moe_dequantize_i8(t(i8, 4, 16), t(f32, 4), bf, src_row=t(i32, n)),
    "moe_swiglu_restore_i8": lambda n: moe.moe_swiglu_restore_i8(t(i8, n, 32), t(f32, n), bf),
    "moe_grouped_gemm_i8": lambda n: moe.moe_grouped_gemm_i8(t(i8, n, 64), t(f32, n), None, t(i32, 3), *W),
    "moe_grouped_gemm_i8 map": lambda n: moe.moe_grouped_gemm_i8(t(i8, 4, 64), t(f32, 4), t(i32, n), t(i32, 3), *W),
    "moe_grouped_ffn_fwd_i8": lambda n: moe.moe_grouped_ffn_fwd_i8(
        t(i8, 4, 64), t(f32, 4), t(i32, n), t(i32, 3), W, W, (t(i8, 2, 64, 32), t(f32, 2, 64))),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("size", [BIG, 1 << 31])
def test_sizes_past_32_bits(monkeypatch, name, size):
    for m in (norm, int8):
        monkeypatch.setattr(m, "_device", lambda x: x.device)
        monkeypatch.setattr(m, "_raw_stream", lambda d: 0)
    with pytest.raises(ValueError, match="32 bits"):
        CALLS[name](size)
