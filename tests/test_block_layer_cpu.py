"""What the layer refuses when it is built, not in its first forward (no GPU: nothing is launched)."""
import pytest
import torch

import moe_expert_layer_router_amd as moe

bf, f32 = torch.bfloat16, torch.float32


def build(H=64, I=64, dt=bf, **kw):
    return moe.MoELayer(16, H, I, 4, 2, 0, 4, dt, "cpu", **kw)


@pytest.mark.parametrize("H,I", [(144, 64), (80, 48), (16, 16), (64, 24)])
def test_an_int8_layer_has_the_routers_widths(H, I):
    with pytest.raises(ValueError, match="multiple of 64"):
        build(H, I, train=False, int8=True)


@pytest.mark.parametrize("H,I", [(64, 16), (128, 144)])
def test_an_int8_layer_takes_any_i_of_sixteens(H, I):
    assert build(H, I, train=False, int8=True).buf["h_perm"].shape == (32, I)


@pytest.mark.parametrize("train", [False, True])
@pytest.mark.parametrize("norm", ["pre_norm", "post_norm"])
def test_norms_that_their_kernels_refuse(norm, train):
    for eps in (0.0, -1.0, float("nan"), float("inf"), 1e-46, 1e300):
        with pytest.raises(ValueError, match=norm):
            build(train=train, **{norm: eps})
    with pytest.raises(moe.MoEError, match="16384"):
        build(H=16448, dt=f32, train=train, **{norm: 1e-6})
    assert build(train=train, **{norm: 1e-6}).buf["y"].shape == (16, 64)
    assert build(train=train, **{norm: torch.finfo(f32).tiny}).buf["y"].shape == (16, 64)
