"""Rows past 2^31 elements whose neighbours differ: the last rows, and those around the 2^31st element, have
the bits that the same rows have alone.  The filler repeats every 61 rows, which divides neither 2^20 rows
(2^31 elements, 2^32 bytes of bf16) nor 2^19, so a row read at an offset cut to 32 bits is another row."""
import pytest
import torch

import moe_expert_layer_router_amd as moe

DEV = torch.device("cuda:0")
pytestmark = pytest.mark.gpu
bf = torch.bfloat16
T, H, PERIOD = (1 << 20) + 1000, 2048, 61
PARTS = [slice(T - 64, T), slice((1 << 20) - 32, (1 << 20) + 32), slice((1 << 19) - 32, (1 << 19) + 32)]


@pytest.fixture(scope="module")
def rows():
    g = torch.Generator(device=DEV).manual_seed(0)
    few = torch.randn((PERIOD, H), generator=g, device=DEV).to(bf)
    x = few.repeat(-(-T // PERIOD), 1)[:T].contiguous()
    x[-64:] = torch.randn((64, H), generator=g, device=DEV).to(bf)
    for r in (T - 1, T - 1000, 1 << 20, 1 << 19):
        assert not torch.equal(x[r], x[r - (1 << 20)]) and not torch.equal(x[r], x[r - (1 << 19)])
    yield x
    del x
    torch.cuda.empty_cache()


def test_norm(rows):
    w = torch.rand(H, device=DEV) + 0.5
    f = moe.moe_norm(rows, w, delta=rows)
    b = moe.moe_norm_bwd(f["n"], f["r"], w, dr=rows)
    for part in PARTS:
        x = rows[part].contiguous()
        e = moe.moe_norm(x, w, delta=x)
        d = moe.moe_norm_bwd(e["n"], e["r"], w, dr=x)
        for a, c in ((f["n"], e["n"]), (f["r"], e["r"]), (b["dx"], d["dx"])):
            assert torch.equal(a[part], c)


def test_combine_norm(rows):
    w = torch.rand(H, device=DEV) + 0.5
    dest = torch.arange(T - 1, -1, -1, device=DEV, dtype=torch.int32)  # token t's row is T - 1 - t
    tw = torch.rand((T, 1), device=DEV) + 0.5
    y = moe.moe_combine_norm(rows, tw, dest, T, w, residual=rows, gate=rows)
    b = moe.moe_combine_norm_bwd(rows, rows, tw, dest, w, gate=rows)
    for tokens in PARTS + [slice(T - s.stop, T - s.start) for s in PARTS]:
        at = slice(T - tokens.stop, T - tokens.start)
        part, own, n = rows[at].contiguous(), rows[tokens].contiguous(), tokens.stop - tokens.start
        back = torch.arange(n - 1, -1, -1, device=DEV, dtype=torch.int32)
        one = tw[tokens].contiguous()
        assert torch.equal(y[tokens], moe.moe_combine_norm(part, one, back, n, w, residual=own, gate=own))
        c = moe.moe_combine_norm_bwd(own, part, one, back, w, gate=own)
        assert torch.equal(b["dy_perm"][at], c["dy_perm"]) and torch.equal(b["d_topk_w"][tokens], c["d_topk_w"])
        assert torch.equal(b["dgate"][tokens], c["dgate"])


@pytest.mark.parametrize("group", [None, 128])
def test_rows_as_8_bit_integers(rows, group):
    q, s = moe.moe_quantize_i8(rows, group=group)
    r = moe.moe_swiglu_restore_i8(q, s, bf)
    for part in PARTS:
        eq, es = moe.moe_quantize_i8(rows[part].contiguous(), group=group)
        assert torch.equal(q[part], eq) and torch.equal(s[part], es)
        src = torch.arange(part.stop - 1, part.start - 1, -1, device=DEV, dtype=torch.int32)
        assert torch.equal(moe.moe_dequantize_i8(q, s, bf, src_row=src), moe.moe_dequantize_i8(eq, es, bf).flip(0))
        e = moe.moe_swiglu_restore_i8(eq, es, bf)
        assert torch.equal(r["gu"][part], e["gu"]) and torch.equal(r["h_perm"][part], e["h_perm"])
    del r
    back = moe.moe_dequantize_i8(q, s, bf)
    for part in PARTS:
        assert torch.equal(back[part], moe.moe_dequantize_i8(q[part].contiguous(), s[part].contiguous(), bf))
    del q, s, back
    torch.cuda.empty_cache()


@pytest.mark.parametrize("E", [1, 200])
def test_product(E):
    """Results past 2^31 elements from 61 rows of x: the parts of a product as one group of their expert."""
    g = torch.Generator(device=DEV).manual_seed(1)
    K, N = 64, 2048
    x = torch.randint(-127, 128, (PERIOD, K), generator=g, device=DEV, dtype=torch.int8)
    xs = torch.rand(PERIOD, generator=g, device=DEV) + 0.5
    w = torch.randint(-127, 128, (E, N, K), generator=g, device=DEV, dtype=torch.int8)
    ws = torch.rand((E, N), generator=g, device=DEV) + 0.5
    src = (torch.arange(T, device=DEV) % PERIOD).to(torch.int32)
    bound = [T * e // E for e in range(E + 1)]
    y = moe.moe_grouped_gemm_i8(x, xs, src, torch.tensor(bound, dtype=torch.int32, device=DEV), w, ws)
    for part in PARTS + [slice(0, 64)]:
        e = max(i for i in range(E) if bound[i] <= part.start)
        stop = min(part.stop, bound[e + 1])
        off = torch.tensor([0, stop - part.start], dtype=torch.int32, device=DEV)
        want = moe.moe_grouped_gemm_i8(x, xs, src[part.start:stop].contiguous(), off, w[e:e + 1].contiguous(),
                                       ws[e:e + 1].contiguous())
        assert torch.equal(y[part.start:stop], want)
