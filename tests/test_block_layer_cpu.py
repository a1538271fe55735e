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
