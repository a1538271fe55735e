"""The layer with norms around it: what it keeps between calls, and its options, alone and together,
against the calls that they are made of (bit for bit: the layer is those calls) and against float64
autograd (the fp32 layer's bar, rel-L2 1e-5: dots of length 64 and sums over 24 tokens err by some 1e-7 of
their size, ten such steps follow one another)."""
import weakref

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


def test_a_captured_gate_gradient_outlives_a_gate_of_the_other_form():
    """A step captured with a gate a token, then an eager step with one an element: the captured step's
    buffer is still the layer's, so a replay writes memory of nobody else."""
    g = torch.Generator(device=DEV).manual_seed(0)
    T, H, I, E, k, eps = 40, 128, 64, 4, 2, 1e-6
    w, ow = weights(g, H, I, E, bf), 1 + rand(g, H, std=0.2)
    x, dy = rand(g, T, H, dt=bf), rand(g, T, H, dt=bf)
    token, full = torch.sigmoid(rand(g, T)), torch.sigmoid(rand(g, T, H)).to(bf)
    layer, other = (moe.MoELayer(T, H, I, E, k, 0, E, bf, DEV, post_norm=eps) for _ in range(2))

    def step(m, gate):
        m.forward(x, *w, post_weight=ow, gate=gate)
        return m.backward(dy, x, *w)["dgate"]

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(layer, token)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            captured = step(layer, token)
    torch.cuda.synchronize()
    for _ in range(3):
        x.copy_(rand(g, T, H, dt=bf))
        got = step(layer, full)
        assert torch.equal(got, step(other, full)) and got.shape == (T, H)
        keep = got.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert any(t is captured for t in layer.buf.values())
        assert torch.equal(captured, step(other, token)) and torch.equal(got, keep)
        assert step(layer, token).data_ptr() == captured.data_ptr()


@pytest.mark.parametrize("form", ["train", "serve", "serve norms", "train post", "train pre"])
def test_a_layer_holds_no_tensor_that_it_does_not_read_again(form):
    """The residual, and in a layer built for the forward alone every input, is its caller's alone once
    forward() is back.  Training with a norm holds what the norm's backward reads."""
    g = torch.Generator(device=DEV).manual_seed(1)
    T, H, I, E, k, eps = 24, 64, 64, 4, 2, 1e-6
    w = weights(g, H, I, E, bf)
    train, pre, post = form.startswith("train"), form in ("serve norms", "train pre"), form in ("serve norms", "train post")
    layer = moe.MoELayer(T, H, I, E, k, 0, E, bf, DEV, train=train, pre_norm=eps if pre else None,
                         post_norm=eps if post else None)
    given = {"x": rand(g, T, H, dt=bf)}
    if pre:
        given["pre_weight"] = torch.ones(H, device=DEV)
    else:
        given["residual"] = rand(g, T, H, dt=bf)
    if post:
        given.update(post_weight=torch.ones(H, device=DEV), gate=torch.rand(T, device=DEV))
    refs = {n: weakref.ref(t) for n, t in given.items()}
    layer.forward(given.pop("x"), *w, **given)
    del given
    held = {n for n, r in refs.items() if r() is not None}
    assert held == ({"train post": {"post_weight", "gate"}, "train pre": {"x", "pre_weight"}}.get(form, set()))


# pre_norm, post_norm, checkpoint, gate, delta, residual
FORMS = {"post": (0, 1, 0, "none", 0, 0), "post, token gate": (0, 1, 0, "token", 0, 1),
         "post, full gate": (0, 1, 0, "full", 0, 1), "pre": (1, 0, 0, "none", 0, 0), "pre, delta": (1, 0, 0, "none", 1, 0),
         "both": (1, 1, 0, "full", 0, 0), "both, delta": (1, 1, 0, "token", 1, 0), "checkpoint, post": (0, 1, 1, "token", 0, 1),
         "checkpoint, pre": (1, 0, 1, "none", 1, 0), "checkpoint, both": (1, 1, 1, "full", 1, 0),
         "checkpoint, both, no delta": (1, 1, 1, "token", 0, 0)}


def inputs(g, form, T, H, dt):
    pre, post, ckpt, gate, delta, residual = FORMS[form]
    a = {"x": rand(g, T, H, dt=dt)}
    if pre:
        a["pre_weight"] = 1 + rand(g, H, std=0.2)
    if post:
        a.update(post_weight=1 + rand(g, H, std=0.2), residual_scale=0.75)
    if gate != "none":
        a["gate"] = torch.sigmoid(rand(g, T)) if gate == "token" else torch.sigmoid(rand(g, T, H)).to(dt)
    if delta:
        a["delta"] = rand(g, T, H, dt=dt)
    if residual:
        a["residual"] = rand(g, T, H, dt=dt)
    return a


def restored(f, offsets, dt, I, H):
    """gu, h_perm and y_perm as their 8-bit codes bring them back."""
    n = offsets[-1:]
    group = next(c for c in (128, 64, 32) if I % c == 0 and H % c == 0)
    q, s = moe.moe_quantize_i8(f["gu"], group=group, nrows=n)
    r = moe.moe_swiglu_restore_i8(q, s, dt, nrows=n)
    q, s = moe.moe_quantize_i8(f["y_perm"], group=group, nrows=n)
    return {**r, "y_perm": moe.moe_dequantize_i8(q, s, dt, nrows=n)}


def chained(form, a, dy, wr, wg, wu, wd, k, eps):
    """The layer's outputs from the library's calls, one after another on one stream."""
    pre, post, ckpt, gate, _, _ = FORMS[form]
    x, (T, H), dt, E = a["x"], a["x"].shape, a["x"].dtype, wr.shape[1]
    rs, gt, r, n = a.get("residual_scale", 1.0), a.get("gate"), a.get("residual"), x
    if pre:
        f = moe.moe_norm(x, a["pre_weight"], eps[0], delta=a.get("delta"))
        r, n = f["r"], f["n"]
    idx, w, _ = moe.moe_route(n, wr, k)
    p = moe.moe_permute(n, idx, E, 0, E)
    f = moe.moe_grouped_ffn_fwd(p["x_perm"], p["offsets"], wg, wu, wd)
    if post:
        y = moe.moe_combine_norm(f["y_perm"], w, p["dest_row"], T, a["post_weight"], eps[1], residual=r, residual_scale=rs,
                                 gate=gt)
    else:
        y = moe.moe_combine_dropout(f["y_perm"], w, p["dest_row"], T, 0.0,
                                    torch.zeros(2, dtype=torch.int64, device=DEV), residual=r)
    if ckpt:
        f = restored(f, p["offsets"], dt, wg.shape[1], H)
    got = {"y": y}
    if post:
        c = moe.moe_combine_norm_bwd(dy, f["y_perm"], w, p["dest_row"], a["post_weight"], eps[1], gate=gt)
        got["dpost_weight"] = c["dweight"]
        if gt is not None:
            got["dgate"] = c["dgate"]
    else:
        c = moe.moe_combine_bwd(dy, f["y_perm"], w, p["dest_row"])
    d = moe.moe_grouped_ffn_bwd(c["dy_perm"], p["x_perm"], f["gu"], f["h_perm"], p["offsets"], wg, wu, wd)
    dx = moe.moe_combine_dx_t(d["dx_perm"], p["dest_row"], c["d_topk_w"], w, idx, moe.moe_router_weight_t(wr))
    rb = moe.moe_route_bwd(c["d_topk_w"], w, idx, n, wr, want_dx=False)
    if pre:
        b = moe.moe_norm_bwd(dx, r, a["pre_weight"], eps[0], dr=dy, dr_scale=rs)
        dx, got["dpre_weight"] = b["dx"], b["dweight"]
    got.update(dx=dx, d_topk_w=c["d_topk_w"], d_logits=rb["d_logits"], dw_router=rb["dw_router"],
               **{n: d[n] for n in ("dw_gate", "dw_up", "dw_down")})
    return got


@pytest.mark.parametrize("dt", [bf, f32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS)
def test_each_form_is_its_calls(form, dt):
    """Two steps with other inputs, the buffers that layers share overwritten between forward and backward."""
    g = torch.Generator(device=DEV).manual_seed(3)
    T, H, I, E, k, eps = 77, 192, 64, 8, 3, (1e-5, 2e-6)
    w = weights(g, H, I, E, dt)
    pre, post, ckpt, *_ = FORMS[form]
    pool = {} if ckpt else None
    layer = moe.MoELayer(T, H, I, E, k, 0, E, dt, DEV, checkpoint=pool, pre_norm=eps[0] if pre else None,
                         post_norm=eps[1] if post else None)
    for _ in range(2):
        a, dy = inputs(g, form, T, H, dt), rand(g, T, H, dt=dt)
        want = chained(form, a, dy, *w, k, eps)
        got = {"y": layer.forward(a["x"], *w, **{n: v for n, v in a.items() if n != "x"}).clone()}
        for t in (pool or {}).values():
            t.fill_(float("nan"))  # whatever another layer left there
        got.update(layer.backward(dy, a["x"], *w))
        assert set(got) == set(want)
        for n in want:
            assert torch.equal(got[n], want[n]), n


def block_ref(a, w, idx, eps, post):
    """The block in float64: a, w the layer's arguments by name."""
    norm = lambda v, weight, e: v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + e) * weight
    r, n = a.get("residual"), a["x"]
    if "pre_weight" in a:
        r = a["x"] + a["delta"] if "delta" in a else a["x"]
        n = norm(r, a["pre_weight"], eps[0])
    weight = torch.softmax(torch.gather(n @ w["router"], 1, idx), dim=1)
    c = 0
    for j in range(idx.shape[1]):
        e = idx[:, j]
        gate = torch.einsum("th,tih->ti", n, w["gate"][e])
        up = torch.einsum("th,tih->ti", n, w["up"][e])
        c = c + weight[:, j, None] * torch.einsum("ti,thi->th", gate * torch.sigmoid(gate) * up, w["down"][e])
    if post:
        c = norm(c, a["post_weight"], eps[1])
        if "gate" in a:
            c = a["gate"].reshape(len(n), -1) * c
    return c if r is None else c + a.get("residual_scale", 1.0) * r


@pytest.mark.parametrize("form", [f for f in FORMS if not f.startswith("checkpoint")])
def test_each_form_against_autograd(form):
    g = torch.Generator(device=DEV).manual_seed(4)
    T, H, I, E, k, eps = 24, 64, 32, 4, 2, (1e-5, 2e-6)
    wr, wg, wu, wd = weights(g, H, I, E, f32)
    a, dy = inputs(g, form, T, H, f32), rand(g, T, H)
    pre, post, *_ = FORMS[form]
    layer = moe.MoELayer(T, H, I, E, k, 0, E, f32, DEV, pre_norm=eps[0] if pre else None, post_norm=eps[1] if post else None)
    y = layer.forward(a["x"], wr, wg, wu, wd, **{n: v for n, v in a.items() if n != "x"})
    got = layer.backward(dy, a["x"], wr, wg, wu, wd)
    leaf = lambda t: t.double().cpu().requires_grad_() if torch.is_tensor(t) else t
    da, dw = {n: leaf(v) for n, v in a.items()}, dict(zip(("router", "gate", "up", "down"), map(leaf, (wr, wg, wu, wd))))
    want = block_ref(da, dw, layer.buf["topk_idx"].long().cpu(), eps, post)
    rel = lambda p, q: float((p.double().cpu() - q).norm() / q.norm())
    assert rel(y, want.detach()) < 1e-5
    leaves = {"dx": da["x"], **{"dw_" + n: t for n, t in dw.items()}}
    for name, of in (("dpre_weight", "pre_weight"), ("dpost_weight", "post_weight"), ("dgate", "gate")):
        if of in da:
            leaves[name] = da[of]
    grads = torch.autograd.grad((want * dy.double().cpu()).sum(), list(leaves.values()))
    for name, v in zip(leaves, grads):
        assert rel(got[name], v) < 1e-5, name


@pytest.mark.parametrize("H,I", [(128, 64), (64, 16), (192, 144)])
@pytest.mark.parametrize("form", ["post, full gate", "pre, delta", "both, delta", "both"])
def test_int8_weights_with_norms_are_their_calls(form, H, I):
    g = torch.Generator(device=DEV).manual_seed(5)
    T, E, k, eps = 60, 8, 2, (1e-5, 2e-6)
    pre, post, *_ = FORMS[form]
    w = weights(g, H, I, E, bf)
    codes = [moe.moe_quantize_i8(t) for t in w[1:]]
    layer = moe.MoELayer(T, H, I, E, k, 0, E, bf, DEV, train=False, int8=True, pre_norm=eps[0] if pre else None,
                         post_norm=eps[1] if post else None)
    for _ in range(2):
        a = inputs(g, form, T, H, bf)
        y = layer.forward(a["x"], w[0], *codes, **{n: v for n, v in a.items() if n != "x"})
        r, n = a.get("residual"), a["x"]
        if pre:
            f = moe.moe_norm(n, a["pre_weight"], eps[0], delta=a.get("delta"))
            r, n = f["r"], f["n"]
        idx, tw, _ = moe.moe_route(n, w[0], k)
        p = moe.moe_permute(n, idx, E, 0, E, copy_rows=False)
        f = moe.moe_grouped_ffn_fwd_i8(*moe.moe_quantize_i8(n), p["src_row"], p["offsets"], *codes)
        if post:
            want = moe.moe_combine_norm(f["y_perm"], tw, p["dest_row"], T, a["post_weight"], eps[1], residual=r,
                                        residual_scale=0.75, gate=a.get("gate"))
        else:
            want = moe.moe_combine_dropout(f["y_perm"], tw, p["dest_row"], T, 0.0,
                                           torch.zeros(2, dtype=torch.int64, device=DEV), residual=r)
        assert torch.equal(y, want)
