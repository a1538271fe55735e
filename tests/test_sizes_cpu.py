"""Sizes that do not fit the library's int32 arguments are refused by the binding, not cut to their
low bits.  Shapes alone are needed: tensors without memory stand in for those on a GPU."""
import pytest
import torch

import moe_expert_layer_router_amd as moe

BIG = (1 << 32) + 5  # 5 in its low 32 bits
bf, f32, i32, i64, u8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


def t(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="meta")


CALLS = {
    "moe_balance_loss": lambda T: moe.moe_balance_loss(t(f32, T, 8), t(i32, T, 2), 0.1),
    "sequences": lambda T: moe.moe_balance_loss(t(f32, 4, 8), t(i32, 4, 2), 0.1, seq_offsets=t(i32, T + 1)),
    "moe_balance_loss_bwd": lambda T: moe.moe_balance_loss_bwd(
        t(f32, T, 8), {"lse": t(f32, T), "counts": t(i32, 1, 8), "tokens": t(i32, 2)}, 2, 0.1),
    "k": lambda T: moe.moe_balance_loss_bwd(
        t(f32, 4, 8), {"lse": t(f32, 4), "counts": t(i32, 1, 8), "tokens": t(i32, 2)}, T, 0.1),
    "moe_route_bwd_add": lambda T: moe.moe_route_bwd_add(
        t(f32, T, 2), t(f32, T, 2), t(i32, T, 2), t(f32, T, 8), t(f32, T, 64), t(f32, 64, 8)),
    "moe_combine_dropout": lambda T: moe.moe_combine_dropout(t(bf, 6, 8), None, t(i32, T), T, 0.1, t(i64, 2)),
    "moe_combine_dropout_bwd": lambda T: moe.moe_combine_dropout_bwd(
        t(bf, T, 8), t(bf, 6, 8), t(f32, T, 1), t(i32, T), 0.1, t(i64, 2)),
    "moe_adapter_fwd": lambda T: moe.moe_adapter_fwd(
        t(bf, T, 8), t(i32, T), t(bf, 2, 16, 8), t(bf, 2, 8, 16), t(bf, T, 8)),
    "x rows": lambda T: moe.moe_adapter_fwd(
        t(bf, T, 8), t(i32, 3), t(bf, 2, 16, 8), t(bf, 2, 8, 16), t(bf, 3, 8), src_row=t(i32, 3)),
    "moe_adapter_bwd": lambda T: moe.moe_adapter_bwd(
        t(bf, T, 8), t(bf, T, 8), t(i32, T), t(bf, 2, 16, 8), t(bf, 2, 8, 16), t(f32, T, 16), None),
    "moe_adapter_rows": lambda T: moe.moe_adapter_rows(t(i32, 5), t(i32, T), t(i32, 4), 2),
    "adapters": lambda T: moe.moe_adapter_rows(t(i32, 5), t(i32, 4), t(i32, 4), T),
    "moe_grouped_ffn_fwd_adapter": lambda T: moe.moe_grouped_ffn_fwd_adapter(
        t(f32, T, 4), None, t(i32, 3), t(i32, T), t(f32, 2, 4, 4), t(f32, 2, 4, 4), t(f32, 2, 4, 4),
        {"up": (t(f32, 2, 8, 4), t(f32, 2, 4, 8))}),
}


@pytest.fixture
def no_gpu(monkeypatch):
    monkeypatch.setattr(moe, "_device", lambda x: x.device)
    monkeypatch.setattr(moe, "_raw_stream", lambda d: 0)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("size", [BIG, 1 << 31])
def test_sizes_past_32_bits(no_gpu, name, size):
    with pytest.raises(ValueError, match="32 bits"):
        CALLS[name](size)


@pytest.mark.parametrize("which", ["x", "y", "dy", "dx"])
def test_pitches_past_32_bits(no_gpu, which):
    wide = torch.empty_strided((3, 8), ((1 << 32) + 8, 1), dtype=bf, device="meta")
    a = {n: wide if n == which else t(bf, 3, 8) for n in ("x", "y", "dy", "dx")}
    w = dict(row_id=t(i32, 3), A=t(bf, 2, 16, 8), B=t(bf, 2, 8, 16))
    with pytest.raises(ValueError, match="32 bits"):
        if which == "y" or which == "x":
            moe.moe_adapter_fwd(a["x"], w["row_id"], w["A"], w["B"], a["y"])
        else:
            moe.moe_adapter_bwd(a["dy"], a["x"], w["row_id"], w["A"], w["B"], t(f32, 3, 16), a["dx"])


@pytest.mark.parametrize("k", [1, 2, 8])
@pytest.mark.parametrize("given", [False, True])
def test_dropout_of_no_tokens(no_gpu, k, given):
    """An empty batch of any number of slots, with the output given or not."""
    out = t(bf, 0, 16) if given else None
    y = moe.moe_combine_dropout(t(bf, 0, 16), t(f32, 0, k), t(i32, 0), 0, 0.1, t(i64, 2), out=out)
    assert y.shape == (0, 16)
    b = moe.moe_combine_dropout_bwd(t(bf, 0, 16), t(bf, 0, 16), t(f32, 0, k), t(i32, 0), 0.1, t(i64, 2))
    assert b["dy_perm"].shape == (0, 16) and b["d_topk_w"].shape == (0, k)
