"""The layer with norms around it, with 8-bit activation checkpoints and with int8 weights.

Bits: each form is the calls it is made of, so it equals them bit for bit.  Gradients of the fp32 layer
with both norms against float64 autograd of the whole block with the kernel's routing: the fp32 layer's
bar (rel-L2 1e-5; dots of length 64 and sums over 24 tokens err by some 1e-7 of their size, ten such steps
follow one another)."""
import numpy as np
import pytest
import torch

import moe_expert_layer_router_amd as moe

DEV = torch.device("cuda:0")
pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def rand(g, *shape, std=1.0, dt=f32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)


def weights(g, H, I, E, dt):
    return (rand(g, H, E, std=H ** -0.5, dt=dt), rand(g, E, I, H, std=H ** -0.5, dt=dt),
            rand(g, E, I, H, std=H ** -0.5, dt=dt), rand(g, E, H, I, std=I ** -0.5, dt=dt))


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_int8_layer_is_its_calls():
    g = torch.Generator(device=DEV).manual_seed(0)
    T, H, I, E, k = 100, 256, 144, 8, 2
    wr, wg, wu, wd = weights(g, H, I, E, bf)
    codes = [moe.moe_quantize_i8(w) for w in (wg, wu, wd)]
    layer = moe.MoELayer(T, H, I, E, k, 2, 7, bf, DEV, train=False, int8=True)
    part = [(q[2:7].contiguous(), s[2:7].contiguous()) for q, s in codes]
    for _ in range(2):
        x = rand(g, T, H, dt=bf)
        y = layer.forward(x, wr, *part)
        idx, w, _ = moe.moe_route(x, wr, k)
        p = moe.moe_permute(x, idx, E, 2, 7, copy_rows=False)
        q, s = moe.moe_quantize_i8(x)
        f = moe.moe_grouped_ffn_fwd_i8(q, s, p["src_row"], p["offsets"], *part)
        assert torch.equal(y, moe.moe_combine(f["y_perm"], w, p["dest_row"], T))
    # and near the exact layer: x, h and the weights in steps of a row's largest / 127.  With rows of normal
    # values (largest 3 to 4 of their size) a step is about 1/35, its rounding 1/120 of the values; h, a
    # product of two, reaches about 10 of its size: 1/45.  Four such errors beside each other: below 1/30.
    full = moe.MoELayer(T, H, I, E, k, 0, E, bf, DEV, train=False, int8=True)
    y = full.forward(x, wr, *codes)
    idx, w, _ = moe.moe_route(x, wr, k)
    want = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    for e in range(E):
        for j in range(k):
            t = torch.nonzero(idx[:, j] == e).squeeze(1)
            a = x[t].double()
            gate, up = a @ wg[e].double().t(), a @ wu[e].double().t()
            want[t] += w[t, j, None].double() * ((gate * torch.sigmoid(gate) * up) @ wd[e].double().t())
    assert rel(y, want) < 1 / 30


def pooled(b, I, H):
    """What the codes of a layer's gu and y_perm restore."""
    n = b["offsets"][-1:]
    grp = 128 if I % 128 == 0 and H % 128 == 0 else 64 if I % 64 == 0 and H % 64 == 0 else 32
    q, s = moe.moe_quantize_i8(b["gu"], group=grp, nrows=n)
    r = moe.moe_swiglu_restore_i8(q, s, b["gu"].dtype, nrows=n)
    q, s = moe.moe_quantize_i8(b["y_perm"], group=grp, nrows=n)
    return r["gu"], r["h_perm"], moe.moe_dequantize_i8(q, s, b["gu"].dtype, nrows=n)


@pytest.mark.parametrize("dt,H,I,lo,hi", [(bf, 256, 128, 0, 8), (bf, 192, 64, 2, 6), (f32, 96, 32, 1, 8)])
def test_checkpointed_layers_share_their_buffers(dt, H, I, lo, hi):
    """Two layers forward, then backward in the other order, with one pool: the gradients are those of plain
    layers whose gu, h_perm and y_perm are what their codes restore."""
    g = torch.Generator(device=DEV).manual_seed(1)
    T, E, k = 90, 8, 3
    ws = [weights(g, H, I, E, dt) for _ in range(2)]
    ws = [(w[0], *(t[lo:hi].contiguous() for t in w[1:])) for w in ws]
    pool = {}
    ckpt = [moe.MoELayer(T, H, I, E, k, lo, hi, dt, DEV, checkpoint=pool) for _ in range(2)]
    assert ckpt[0].buf["gu"] is ckpt[1].buf["gu"] and set(pool) == {"x_perm", "gu", "h_perm", "y_perm"}
    plain = [moe.MoELayer(T, H, I, E, k, lo, hi, dt, DEV) for _ in range(2)]
    for step in range(2):
        x, dy = rand(g, T, H, dt=dt), rand(g, T, H, dt=dt)
        xs, ys = [x], []
        for a, b, w in zip(ckpt, plain, ws):
            y = a.forward(xs[-1], *w)
            assert torch.equal(y, b.forward(xs[-1], *w))
            xs.append(y.clone())
        torch.cuda.synchronize()
        for t in pool.values():
            t.fill_(float("nan"))  # whatever another layer left there
        d = dy
        for i in (1, 0):
            got = {n: v.clone() for n, v in ckpt[i].backward(d, xs[i], *ws[i]).items()}
            R = int(plain[i].buf["offsets"][-1])
            for name, v in zip(("gu", "h_perm", "y_perm"), pooled(plain[i].buf, I, H)):
                plain[i].buf[name][:R] = v[:R]
            want = plain[i].backward(d, xs[i], *ws[i])
            for n in want:
                assert torch.equal(got[n], want[n]), (i, n)
            d = got["dx"]


def block_ref(x, delta, pw, ow, gate, rs, wr, wg, wu, wd, idx, eps):
    r = x + delta
    norm = lambda v, w: v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps) * w
    n = norm(r, pw)
    z = torch.gather(n @ wr, 1, idx)
    w = torch.softmax(z, dim=1)
    c = 0
    for j in range(idx.shape[1]):
        e = idx[:, j]
        a = torch.einsum("th,tih->ti", n, wg[e])
        u = torch.einsum("th,tih->ti", n, wu[e])
        c = c + w[:, j, None] * torch.einsum("ti,thi->th", a * torch.sigmoid(a) * u, wd[e])
    return rs * r + gate.reshape(len(x), -1) * norm(c, ow)


@pytest.mark.parametrize("gate_kind", ["token", "full"])
def test_block_gradients_against_autograd(gate_kind):
    g = torch.Generator(device=DEV).manual_seed(2)
    T, H, I, E, k, eps, rs = 24, 64, 32, 4, 2, 1e-5, 0.75
    wr, wg, wu, wd = weights(g, H, I, E, f32)
    x, delta, dy = rand(g, T, H), rand(g, T, H), rand(g, T, H)
    pw, ow = 1 + rand(g, H, std=0.2), 1 + rand(g, H, std=0.2)
    gate = torch.sigmoid(rand(g, T)) if gate_kind == "token" else torch.sigmoid(rand(g, T, H))
    layer = moe.MoELayer(T, H, I, E, k, 0, E, f32, DEV, pre_norm=eps, post_norm=eps)
    y = layer.forward(x, wr, wg, wu, wd, delta=delta, pre_weight=pw, post_weight=ow, gate=gate, residual_scale=rs)
    got = layer.backward(dy, x, wr, wg, wu, wd)
    idx = layer.buf["topk_idx"].long().cpu()
    args = [t.double().cpu().requires_grad_() for t in (x, delta, pw, ow, gate, wr, wg, wu, wd)]
    a = args
    want = block_ref(a[0], a[1], a[2], a[3], a[4], rs, a[5], a[6], a[7], a[8], idx, eps)
    assert rel(y.cpu(), want.detach()) < 1e-5
    grads = torch.autograd.grad((want * dy.double().cpu()).sum(), args)
    for name, w in zip(("dx", "dx", "dpre_weight", "dpost_weight", "dgate", "dw_router", "dw_gate", "dw_up", "dw_down"), grads):
        assert rel(got[name].cpu(), w) < 1e-5, name


@pytest.mark.parametrize("fp8", [False, True])
def test_norms_and_checkpoint_in_a_graph(fp8):
    """A bf16 block with both norms, auxiliary losses and (not FP8) a checkpoint: the layer's calls one by
    one give its bits, and a captured step repeats them over new inputs."""
    g = torch.Generator(device=DEV).manual_seed(3)
    T, H, I, E, k, eps, rs = 130, 256, 128, 8, 2, 1e-6, 0.5
    w = weights(g, H, I, E, bf)
    pw, ow, gate = 1 + rand(g, H, std=0.2), 1 + rand(g, H, std=0.2), torch.sigmoid(rand(g, T))
    x, delta, dy = (rand(g, T, H, dt=bf) for _ in range(3))
    make = lambda: moe.MoELayer(T, H, I, E, k, 0, E, bf, DEV, fp8=fp8, pre_norm=eps, post_norm=eps, balance_coef=0.01,
                                checkpoint=None if fp8 else {})
    layer, eager = make(), make()

    def step(m):
        y = m.forward(x, *w, delta=delta, pre_weight=pw, post_weight=ow, gate=gate, residual_scale=rs)
        return [y, *m.backward(dy, x, *w).values()]

    # forward from its calls
    y = step(eager)[0]
    n = moe.moe_norm(x, pw, eps, delta=delta)
    assert torch.equal(eager.buf["n"], n["n"])
    if fp8:  # (a checkpoint's backward leaves restored rows in y_perm)
        want = moe.moe_combine_norm(eager.buf["y_perm"], eager.buf["topk_w"], eager.buf["dest_row"], T, ow, eps,
                                    residual=n["r"], residual_scale=rs, gate=gate)
        assert torch.equal(y, want)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(layer)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs = step(layer)
    for _ in range(3):
        for t in (x, delta, dy):
            t.copy_(rand(g, T, H, dt=bf))
        want = [t.clone() for t in step(eager)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_pre_norm_alone_with_dropout_and_serving():
    g = torch.Generator(device=DEV).manual_seed(4)
    T, H, I, E, k, eps = 60, 128, 64, 4, 2, 1e-6
    w = weights(g, H, I, E, bf)
    pw, x = 1 + rand(g, H, std=0.2), rand(g, T, H, dt=bf)
    rng = torch.tensor([5, 7], dtype=torch.int64, device=DEV)
    layer = moe.MoELayer(T, H, I, E, k, 0, E, bf, DEV, pre_norm=eps, dropout=0.2)
    ref = moe.MoELayer(T, H, I, E, k, 0, E, bf, DEV, dropout=0.2)
    y = layer.forward(x, *w, rng=rng, pre_weight=pw)
    n = moe.moe_norm(x, pw, eps)["n"]
    assert torch.equal(y, ref.forward(n, *w, rng=rng, residual=x))
    dy = rand(g, T, H, dt=bf)
    got, want = layer.backward(dy, x, *w), ref.backward(dy, n, *w)
    b = moe.moe_norm_bwd(want["dx"], x, pw, eps, dr=dy)
    assert torch.equal(got["dx"], b["dx"]) and torch.equal(got["dpre_weight"], b["dweight"])
    serve = moe.MoELayer(T, H, I, E, k, 0, E, bf, DEV, train=False, pre_norm=eps, post_norm=eps, int8=True)
    codes = [moe.moe_quantize_i8(t) for t in w[1:]]
    y = serve.forward(x, w[0], *codes, pre_weight=pw, post_weight=pw, residual_scale=1.5)
    assert torch.isfinite(y.float()).all() and y.shape == (T, H)


def test_layer_refusals():
    mk = lambda **kw: moe.MoELayer(16, 64, 64, 4, 2, kw.pop("lo", 0), kw.pop("hi", 4), kw.pop("dt", bf), DEV, **kw)
    for kw in (dict(int8=True), dict(int8=True, train=False, dt=f32), dict(int8=True, train=False, adapters=True),
               dict(checkpoint={}, train=False), dict(checkpoint={}, fp8=True), dict(pre_norm=1e-6, lo=1),
               dict(post_norm=1e-6, hi=3), dict(post_norm=1e-6, dropout=0.1)):
        with pytest.raises(ValueError):
            mk(**kw)
    pool = {}
    mk(checkpoint=pool)
    with pytest.raises(ValueError, match="pool"):
        moe.MoELayer(17, 64, 64, 4, 2, 0, 4, bf, DEV, checkpoint=pool)
    g = torch.Generator(device=DEV).manual_seed(5)
    w, x, v = weights(g, 64, 64, 4, bf), rand(g, 16, 64, dt=bf), torch.ones(64, device=DEV)
    plain, pre, post = mk(), mk(pre_norm=1e-6), mk(post_norm=1e-6)
    for layer, kw in ((plain, dict(pre_weight=v)), (plain, dict(delta=x)), (plain, dict(gate=v)), (plain, dict(residual_scale=2.0)),
                      (pre, dict()), (pre, dict(pre_weight=v, residual=x)), (post, dict()), (post, dict(post_weight=v, delta=x)),
                      (post, dict(post_weight=v, gate=v))):
        with pytest.raises(ValueError):
            layer.forward(x, *w, **kw)
