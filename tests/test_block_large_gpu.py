"""The norms, the 8-bit rows and the int8 products past 2^31 elements: the last rows have the bits that
the same rows have alone."""
import pytest
import torch

import moe_expert_layer_router_amd as moe

DEV = torch.device("cuda:0")
pytestmark = pytest.mark.gpu
bf = torch.bfloat16
T, H, LAST = (1 << 20) + 1000, 2048, 64  # 2^31 + 2 million elements


@pytest.fixture(scope="module")
def rows():
    g = torch.Generator(device=DEV).manual_seed(0)
    few = torch.randn((LAST, H), generator=g, device=DEV).to(bf)
    x = few.repeat(-(-T // LAST), 1)[:T].contiguous()
    yield x
    del x
    torch.cuda.empty_cache()


def test_norm(rows):
    w = torch.rand(H, device=DEV) + 0.5
    f = moe.moe_norm(rows, w, delta=rows)
    b = moe.moe_norm_bwd(f["n"], f["r"], w, dr=rows)
    e = moe.moe_norm(rows[-LAST:], w, delta=rows[-LAST:])
    d = moe.moe_norm_bwd(e["n"], e["r"], w, dr=rows[-LAST:])
    for a, c in ((f["n"], e["n"]), (f["r"], e["r"]), (b["dx"], d["dx"])):
        assert torch.equal(a[-LAST:], c)


def test_combine_norm(rows):
    w = torch.rand(H, device=DEV) + 0.5
    dest = torch.arange(T - 1, -1, -1, device=DEV, dtype=torch.int32)
    tw = torch.full((T, 1), 0.5, device=DEV)
    y = moe.moe_combine_norm(rows, tw, dest, T, w, residual=rows)
    b = moe.moe_combine_norm_bwd(rows, rows, tw, dest, w)
    for t0, r0 in ((T - LAST, 0), (0, T - LAST)):  # the last tokens with the first grouped rows, and the reverse
        part = rows[r0:r0 + LAST].contiguous()
        back = torch.arange(LAST - 1, -1, -1, device=DEV, dtype=torch.int32)
        one = torch.full((LAST, 1), 0.5, device=DEV)
        assert torch.equal(y[t0:t0 + LAST], moe.moe_combine_norm(part, one, back, LAST, w, residual=rows[t0:t0 + LAST]))
        c = moe.moe_combine_norm_bwd(rows[t0:t0 + LAST], part, one, back, w)
        assert torch.equal(b["dy_perm"][r0:r0 + LAST], c["dy_perm"])
        assert torch.equal(b["d_topk_w"][t0:t0 + LAST], c["d_topk_w"])


def test_rows_as_8_bit_integers(rows):
    tail = rows[-LAST:].contiguous()
    for group in (None, 128):
        q, s = moe.moe_quantize_i8(rows, group=group)
        eq, es = moe.moe_quantize_i8(tail, group=group)
        assert torch.equal(q[-LAST:], eq) and torch.equal(s[-LAST:], es)
        src = torch.arange(T - 1, T - 1 - LAST, -1, device=DEV, dtype=torch.int32)
        assert torch.equal(moe.moe_dequantize_i8(q, s, bf, src_row=src), moe.moe_dequantize_i8(eq, es, bf).flip(0))
        r, e = moe.moe_swiglu_restore_i8(q, s, bf), moe.moe_swiglu_restore_i8(eq, es, bf)
        assert torch.equal(r["gu"][-LAST:], e["gu"]) and torch.equal(r["h_perm"][-LAST:], e["h_perm"])
        del q, s, r
        torch.cuda.empty_cache()


@pytest.mark.parametrize("E", [1, 200])
def test_product(E):
    """Results past 2^31 elements, from a few rows of x, in tiles of both heights' rule."""
    g = torch.Generator(device=DEV).manual_seed(1)
    K, N = 64, 2048
    x = torch.randint(-127, 128, (LAST, K), generator=g, device=DEV, dtype=torch.int8)
    xs = torch.rand(LAST, generator=g, device=DEV) + 0.5
    w = torch.randint(-127, 128, (E, N, K), generator=g, device=DEV, dtype=torch.int8)
    ws = torch.rand((E, N), generator=g, device=DEV) + 0.5
    src = (torch.arange(T, device=DEV) % LAST).to(torch.int32)
    off = (torch.arange(E + 1, device=DEV) * T // E).to(torch.int32)
    y = moe.moe_grouped_gemm_i8(x, xs, src, off, w, ws)
    last = torch.tensor([0, LAST], dtype=torch.int32, device=DEV)
    want = moe.moe_grouped_gemm_i8(x, xs, src[-LAST:].contiguous(), last, w[-1:].contiguous(), ws[-1:].contiguous())
    assert torch.equal(y[-LAST:], want)
    first = moe.moe_grouped_gemm_i8(x, xs, src[:LAST].contiguous(), last, w[:1].contiguous(), ws[:1].contiguous())
    assert torch.equal(y[:LAST], first)
