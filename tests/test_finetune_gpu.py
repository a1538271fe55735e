"""The operators around the layer used together, as a fine-tuning step and a serving forward use
them: MoELayer with auxiliary losses, dropout, residual and adapters, and a step written with the
calls themselves, against float64 autograd (routing taken from the GPU).

fp32 tolerances: those of the fp32 layer (max-abs 1e-4, rel-L2 1e-5); gradients that sum over all
tokens are held to the rel-L2 alone.  bf16 layers equal, bit for bit, the calls they are made of."""
import numpy as np
import pytest
import torch

import moe_expert_layer_router_amd as moe
from workloads import EP_SHARE, TINY, make_inputs
from test_dropout import keep_mask

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
f64 = torch.float64


def inputs(w, dtype):
    inp = make_inputs(w)
    return {n: torch.from_numpy(np.ascontiguousarray(inp[n])).to(DEV).to(dtype).contiguous()
            for n in ("x", "w_router", "w_gate", "w_up", "w_down")}


def close(got, ref, name, elementwise=True):
    d, r = (got.double().cpu() - ref.cpu()), ref.cpu()
    rel = float(d.norm() / max(float(r.norm()), 1e-30))
    print(f"  {name}: max-abs {float(d.abs().max()):.2e} rel-L2 {rel:.2e}", flush=True)
    assert torch.isfinite(got).all() and rel <= 1e-5
    assert not elementwise or float(d.abs().max()) <= 1e-4


def definition(t, idx, lo, hi, keep, scale, residual, off, live, cb, cz, ad=None):
    """The layer in float64 on the given choices: y and the auxiliary loss; ad: (A, B, s) of the
    down projection, one adapter for each local expert."""
    x, wr, wg, wu, wd = (t[n] for n in ("x", "w_router", "w_gate", "w_up", "w_down"))
    z = x @ wr
    w = torch.softmax(z.gather(1, idx), dim=1)
    y = torch.zeros_like(x)
    for e in range(lo, hi):
        tok, slot = torch.nonzero(idx == e, as_tuple=True)
        xe = x[tok]
        h = torch.nn.functional.silu(xe @ wg[e - lo].t()) * (xe @ wu[e - lo].t())
        o = h @ wd[e - lo].t()
        if ad is not None:
            o = o + ad[2][e - lo] * (h @ ad[0][e - lo].t()) @ ad[1][e - lo].t()
        y = y.index_add(0, tok, w[tok, slot, None] * o)
    y = residual + keep * scale * y
    p, lse = torch.softmax(z, dim=1), torch.logsumexp(z, dim=1)
    N, E, k = int(live.sum()), z.shape[1], idx.shape[1]
    bal = 0.0
    for s in range(len(off) - 1):
        rows = torch.arange(off[s], off[s + 1])
        rows = rows[live[rows]]
        if len(rows):
            c = torch.bincount(idx[rows].reshape(-1), minlength=E).to(f64)
            bal = bal + E / (k * N * len(rows)) * (c * p[rows].sum(dim=0)).sum()
    return y, cb * bal + cz * (lse[live] ** 2).sum() / N


@pytest.mark.parametrize("lo,hi", [(0, 8), (2, 6)])
def test_training_step_of_the_layer_fp32(lo, hi):
    w = TINY.scaled(name="t", T=150, e_lo=lo, e_hi=hi)
    t = inputs(w, torch.float32)
    p, cb, cz, seed, offset = 0.3, 0.05, 0.01, 1234567, 89
    off = np.array([0, 40, 40, 131], np.int32)
    g = torch.Generator().manual_seed(5)
    live = (torch.rand(w.T, generator=g) > 0.2) & (torch.arange(w.T) < 131)
    residual, dy = torch.randn(w.T, w.H, generator=g), torch.randn(w.T, w.H, generator=g)
    layer = moe.MoELayer(w.T, w.H, w.I, w.E, w.k, lo, hi, torch.float32, DEV, balance_coef=cb, z_coef=cz,
                         max_sequences=3, dropout=p)
    rng = torch.tensor([seed, offset], dtype=torch.int64, device=DEV)
    a = (t["x"], t["w_router"], t["w_gate"], t["w_up"], t["w_down"])
    y = layer.forward(*a, residual=residual.to(DEV), rng=rng, seq_offsets=torch.from_numpy(off).to(DEV),
                      token_mask=live.to(torch.uint8).to(DEV))
    d_aux = torch.tensor([1.5], device=DEV)
    grads = layer.backward(dy.to(DEV), *a, d_aux=d_aux)
    torch.cuda.synchronize()
    ref = {n: v.double().cpu().requires_grad_() for n, v in t.items()}
    keep = torch.from_numpy(keep_mask(seed, offset, w.T, w.H, p)).to(f64)
    idx = layer.buf["topk_idx"].cpu().long()
    yr, aux = definition(ref, idx, lo, hi, keep, 1 / (1 - p), residual.double(), off, live,
                         float(np.float32(cb)), float(np.float32(cz)))
    ((yr * dy.double()).sum() + 1.5 * aux).backward()
    close(y, yr.detach(), "y")
    close(layer.buf["aux_loss"][2:], aux.detach().reshape(1), "aux_loss")
    close(grads["dx"], ref["x"].grad, "dx")
    for n, m in (("dw_router", "w_router"), ("dw_gate", "w_gate"), ("dw_up", "w_up"), ("dw_down", "w_down")):
        close(grads[n], ref[m].grad, n, elementwise=False)


def test_step_of_calls_with_adapters_fp32():
    """route, permute, FFN, adapters on the down projection, dropout, loss; and all the way back."""
    w = TINY.scaled(name="t", T=200)
    t = inputs(w, torch.float32)
    T, H, I, E, k = w.T, w.H, w.I, w.E, w.k
    p, seed, offset = 0.25, 99, 3
    g = torch.Generator().manual_seed(6)
    A = (torch.randn(E, 8, I, generator=g) * 0.2)
    B = (torch.randn(E, H, 8, generator=g) * 0.2)
    s = torch.rand(E, generator=g) + 0.5
    residual, dy = torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)
    Ad, Bd, sd = A.to(DEV), B.to(DEV), s.to(DEV)
    rng = torch.tensor([seed, offset], dtype=torch.int64, device=DEV)
    idx, gate, logits = moe.moe_route(t["x"], t["w_router"], k, want_logits=True)
    perm = moe.moe_permute(t["x"], idx, E, 0, E)
    f = moe.moe_grouped_ffn_fwd(perm["x_perm"], perm["offsets"], t["w_gate"], t["w_up"], t["w_down"])
    row_id = moe.moe_adapter_rows(perm["offsets"], perm["src_row"],
                                  torch.zeros(T, dtype=torch.int32, device=DEV), 1)
    v = moe.moe_adapter_fwd(f["h_perm"], row_id, Ad, Bd, f["y_perm"], scale=sd, want_v=True)
    y = moe.moe_combine_dropout(f["y_perm"], gate, perm["dest_row"], T, p, rng, residual=residual.to(DEV))
    aux = moe.moe_balance_loss(logits, idx, 0.1, 0.02)
    c = moe.moe_combine_dropout_bwd(dy.to(DEV), f["y_perm"], gate, perm["dest_row"], p, rng)
    dh = torch.zeros_like(f["h_perm"])
    ad = moe.moe_adapter_bwd(c["dy_perm"], f["h_perm"], row_id, Ad, Bd, v, dh, scale=sd)
    d_add = moe.moe_balance_loss_bwd(logits, aux, k, 0.1, 0.02)
    r = moe.moe_route_bwd_add(c["d_topk_w"], gate, idx, d_add, t["x"], t["w_router"])
    torch.cuda.synchronize()
    ref = {n: x.double().cpu().requires_grad_(n == "w_router") for n, x in t.items()}
    Ar, Br = A.double().requires_grad_(), B.double().requires_grad_()
    keep = torch.from_numpy(keep_mask(seed, offset, T, H, p)).to(f64)
    yr, ar = definition(ref, idx.cpu().long(), 0, E, keep, 1 / (1 - p), residual.double(), [0, T],
                        torch.ones(T, dtype=torch.bool), float(np.float32(0.1)), float(np.float32(0.02)),
                        ad=(Ar, Br, s.double()))
    ((yr * dy.double()).sum() + ar).backward()
    close(y, yr.detach(), "y")
    close(aux["loss"][2:], ar.detach().reshape(1), "loss")
    close(ad["dA"], Ar.grad, "dA", elementwise=False)
    close(ad["dB"], Br.grad, "dB", elementwise=False)
    close(r["dw_router"], ref["w_router"].grad, "dw_router", elementwise=False)
    # dh of the adapters alone: s A^T (B^T dy), row by row
    sorted_e = row_id.cpu().long()
    want = s.double()[sorted_e, None] * torch.einsum(
        "rn,rnj,rji->ri", c["dy_perm"].double().cpu(), B.double()[sorted_e], A.double()[sorted_e])
    close(dh, want, "dh")


@pytest.mark.parametrize("fp8", [False, True])
def test_bf16_layer_is_made_of_its_calls(fp8):
    """Dropout, residual and losses leave the rest of the layer as it is, and a captured step
    replays with new dropout numbers."""
    w = EP_SHARE.scaled(name="l", T=300, H=256, I=128, E=64, k=4, e_lo=8, e_hi=40)
    t = inputs(w, torch.bfloat16)
    a = (t["x"], t["w_router"], t["w_gate"], t["w_up"], t["w_down"])
    shape = (w.T, w.H, w.I, w.E, w.k, w.e_lo, w.e_hi, torch.bfloat16, DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    residual = torch.randn(w.T, w.H, generator=g, device=DEV).bfloat16()
    dy = torch.randn(w.T, w.H, generator=g, device=DEV).bfloat16()
    off = torch.tensor([0, 100, 300], dtype=torch.int32, device=DEV)
    layer = moe.MoELayer(*shape, fp8=fp8, balance_coef=0.1, z_coef=0.01, max_sequences=2, dropout=0.2)
    plain = moe.MoELayer(*shape, fp8=fp8)
    rng = torch.tensor([7, 0], dtype=torch.int64, device=DEV)

    def step():
        layer.forward(*a, residual=residual, rng=rng, seq_offsets=off)
        layer.backward(dy, *a)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        rng[1] += 1
    before = None
    for i in range(3):
        now = rng.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: layer.buf[n].clone() for n in ("y", "dx", "dw_router", "dw_gate", "dw_down", "d_logits", "aux_loss")}
        # the same step by hand, on the plain layer's buffers
        plain.forward(*a)
        b = plain.buf
        y = moe.moe_combine_dropout(b["y_perm"], b["topk_w"], b["dest_row"], w.T, 0.2, now, residual=residual)
        assert torch.equal(y, got["y"])
        f = moe.moe_balance_loss(b["logits"], b["topk_idx"], 0.1, 0.01, seq_offsets=off)
        assert torch.equal(f["loss"], got["aux_loss"])
        R = int(b["offsets"][-1])
        c = moe.moe_combine_dropout_bwd(dy, b["y_perm"], b["topk_w"], b["dest_row"], 0.2, now)
        assert torch.equal(c["dy_perm"][:R], layer.buf["dy_perm"][:R])
        d = moe.moe_balance_loss_bwd(b["logits"], f, w.k, 0.1, 0.01, seq_offsets=off)
        r = moe.moe_route_bwd_add(c["d_topk_w"], b["topk_w"], b["topk_idx"], d, t["x"], t["w_router"])
        assert torch.equal(r["d_logits"], got["d_logits"]) and torch.equal(r["dw_router"], got["dw_router"])
        dx = moe.moe_combine(layer.buf["dx_perm"], None, b["dest_row"], w.T, addend=r["dx_router"])
        assert torch.equal(dx, got["dx"])
        assert before is None or not torch.equal(before, got["y"])
        before = got["y"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_forward_with_adapters(dtype):
    """Three requests' adapters on the three projections: rows without one as in the plain layer,
    the others near the definition (bf16: within the layer's rel-L2 of 5e-3)."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    w = EP_SHARE.scaled(name="l", T=190, H=256, I=128, E=16, k=4, e_lo=4, e_hi=12, dtype=dtype)
    t = inputs(w, dt)
    a = (t["x"], t["w_router"], t["w_gate"], t["w_up"], t["w_down"])
    E_l, n, rank = 8, 3, 16
    g = torch.Generator(device=DEV).manual_seed(2)
    rnd = lambda *s, std: (torch.randn(s, generator=g, device=DEV) * std).to(dt)
    ad = dict(n=n, token_adapter=torch.randint(-1, n, (w.T,), generator=g, device=DEV, dtype=torch.int32),
              gate=(rnd(n, E_l, rank, w.H, std=0.05), rnd(n, E_l, w.I, rank, std=0.2)),
              up=(rnd(n, E_l, rank, w.H, std=0.05), rnd(n, E_l, w.I, rank, std=0.2)),
              down=(rnd(n, E_l, rank, w.I, std=0.05), rnd(n, E_l, w.H, rank, std=0.2)),
              scale=torch.rand(n, E_l, generator=g, device=DEV) + 0.5)
    shape = (w.T, w.H, w.I, w.E, w.k, w.e_lo, w.e_hi, dt, DEV)
    layer, plain = moe.MoELayer(*shape, train=False, adapters=True), moe.MoELayer(*shape, train=False)
    y, y0 = layer.forward(*a, adapters=ad), plain.forward(*a)
    torch.cuda.synchronize()
    none = ad["token_adapter"] < 0
    assert none.any() and torch.equal(y[none], y0[none]) and not torch.equal(y, y0)
    idx, gate = layer.buf["topk_idx"].long().cpu(), layer.buf["topk_w"].double().cpu()
    d = lambda x: x.double().cpu()
    ref = torch.zeros(w.T, w.H, dtype=f64)
    x, who = d(t["x"]), ad["token_adapter"].cpu()
    for tok in range(w.T):
        for j in range(w.k):
            e = int(idx[tok, j]) - w.e_lo
            if not 0 <= e < E_l:
                continue
            q = int(who[tok])
            low = lambda name, v: 0 if q < 0 else d(ad["scale"][q, e]) * d(ad[name][1][q, e]) @ (d(ad[name][0][q, e]) @ v)
            gg = d(t["w_gate"][e]) @ x[tok] + low("gate", x[tok])
            uu = d(t["w_up"][e]) @ x[tok] + low("up", x[tok])
            h = torch.nn.functional.silu(gg) * uu
            ref[tok] += gate[tok, j] * (d(t["w_down"][e]) @ h + low("down", h))
    rel = float((d(y) - ref).norm() / ref.norm())
    print("  rel-L2", rel, flush=True)
    assert rel <= (5e-3 if dtype == "bf16" else 1e-5)
    # the plain forward of the same layer, and one projection alone
    assert torch.equal(layer.forward(*a), y0)
    only = {k_: v for k_, v in ad.items() if k_ not in ("gate", "up")}
    assert not torch.equal(layer.forward(*a, adapters=only), y0)


def test_refusals():
    with pytest.raises(ValueError, match="dropout"):
        moe.MoELayer(8, 64, 64, 8, 2, 0, 8, torch.float32, DEV, dropout=1.0)
    with pytest.raises(ValueError, match="adapters"):
        moe.MoELayer(8, 64, 64, 8, 2, 0, 8, torch.bfloat16, DEV, adapters=True)
    w = TINY.scaled(name="t", T=8)
    t = inputs(w, torch.float32)
    a = (t["x"], t["w_router"], t["w_gate"], t["w_up"], t["w_down"])
    shape = (w.T, w.H, w.I, w.E, w.k, 0, 8, torch.float32, DEV)
    with pytest.raises(ValueError, match="rng"):
        moe.MoELayer(*shape, dropout=0.1).forward(*a)
    with pytest.raises(ValueError, match="without adapters"):
        moe.MoELayer(*shape).forward(*a, adapters={})
    with pytest.raises(ValueError, match="logits"):
        moe.MoELayer(*shape, balance_coef=0.1).forward(*a, save_logits=False)
    with pytest.raises(ValueError, match="sequences"):
        moe.MoELayer(*shape, balance_coef=0.1).forward(*a, seq_offsets=torch.zeros(3, dtype=torch.int32, device=DEV))
    p = moe.moe_permute(t["x"], torch.zeros((8, 1), dtype=torch.int32, device=DEV), 8, 0, 8)
    with pytest.raises(ValueError, match="gate, up, down"):
        moe.moe_grouped_ffn_fwd_adapter(p["x_perm"], None, p["offsets"], p["src_row"], *a[2:], {})


def test_one_sequence_in_a_layer_for_several():
    """Without seq_offsets all tokens are one sequence, in a layer built for more as well."""
    w = TINY.scaled(name="t", T=90)
    t = inputs(w, torch.float32)
    a = (t["x"], t["w_router"], t["w_gate"], t["w_up"], t["w_down"])
    shape = (w.T, w.H, w.I, w.E, w.k, 0, 8, torch.float32, DEV)
    one, four = (moe.MoELayer(*shape, balance_coef=0.1, z_coef=0.02, max_sequences=n) for n in (1, 4))
    mask = (torch.arange(w.T, device=DEV) % 5 != 0).to(torch.uint8)
    dy = torch.ones(w.T, w.H, device=DEV)
    got = []
    for layer in (one, four):
        layer.forward(*a, token_mask=mask)
        grads = layer.backward(dy, *a)
        got.append([grads["d_logits"], grads["dx"], layer.buf["aux_loss"], layer.buf["aux_counts"][0],
                    layer.buf["aux_prob_sum"][0]])
    for u, v in zip(*got):
        assert torch.equal(u, v)
    assert not four.buf["aux_counts"][1:].any() and not four.buf["aux_prob_sum"][1:].any()
    assert four.buf["aux_tokens"].tolist() == [72, 0, 0, 0, 72]
    with pytest.raises(ValueError, match="sequences"):
        four.forward(*a, seq_offsets=torch.tensor([0, w.T], dtype=torch.int32, device=DEV))


def test_projections_without_adapters():
    """A projection given as None is one that is not given, first or last; all of them None is refused."""
    w = EP_SHARE.scaled(name="l", T=33, H=128, I=64, E=8, k=2, e_lo=0, e_hi=8)
    t = inputs(w, torch.bfloat16)
    a = (t["x"], t["w_router"], t["w_gate"], t["w_up"], t["w_down"])
    g = torch.Generator(device=DEV).manual_seed(3)
    rnd = lambda *s: (torch.randn(s, generator=g, device=DEV) * 0.2).bfloat16()
    up = (rnd(2, 8, 8, w.H), rnd(2, 8, w.I, 8))
    who = torch.randint(-1, 2, (w.T,), generator=g, device=DEV, dtype=torch.int32)
    layer = moe.MoELayer(w.T, w.H, w.I, w.E, w.k, 0, 8, torch.bfloat16, DEV, train=False, adapters=True)
    plain = layer.forward(*a).clone()
    want = layer.forward(*a, adapters=dict(n=2, token_adapter=who, up=up)).clone()
    got = layer.forward(*a, adapters=dict(n=2, token_adapter=who, gate=None, up=up, down=None))
    assert torch.equal(got, want) and not torch.equal(got, plain)
    p = moe.moe_permute(t["x"], layer.buf["topk_idx"], 8, 0, 8)
    rows = moe.moe_adapter_rows(p["offsets"], p["src_row"], who, 2)
    call = lambda ad: moe.moe_grouped_ffn_fwd_adapter(p["x_perm"], None, p["offsets"], rows, *a[2:], ad)["y_perm"]
    flat = tuple(u.reshape(16, *u.shape[2:]) for u in up)
    n = int(p["offsets"][-1])
    assert torch.equal(call({"gate": None, "up": flat})[:n], call({"up": flat})[:n])
    with pytest.raises(ValueError, match="gate, up, down"):
        call({"gate": None, "down": None})
    with pytest.raises(ValueError, match="gate, up, down"):
        layer.forward(*a, adapters=dict(n=2, token_adapter=who))


def test_misnamed_projections_are_refused():
    """A key of the adapters that means nothing would leave its projection without them, in silence."""
    w = TINY.scaled(name="t", T=8)
    t = inputs(w, torch.float32)
    a = (t["x"], t["w_router"], t["w_gate"], t["w_up"], t["w_down"])
    layer = moe.MoELayer(w.T, w.H, w.I, w.E, w.k, 0, 8, torch.float32, DEV, train=False, adapters=True)
    who = torch.zeros(w.T, dtype=torch.int32, device=DEV)
    up = (torch.zeros(1, 8, 8, w.H, device=DEV), torch.zeros(1, 8, w.I, 8, device=DEV))
    layer.forward(*a, adapters=dict(n=1, token_adapter=who, up=up))
    for wrong in (dict(gat=up), dict(w_down=up), dict(scales=torch.ones(1, 8, device=DEV))):
        with pytest.raises(ValueError, match=next(iter(wrong))):
            layer.forward(*a, adapters=dict(n=1, token_adapter=who, up=up, **wrong))
