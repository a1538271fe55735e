"""What the norms around the MoE expert layer, its 8-bit activation checkpoints and its int8 products cost.

Four operators, each on the sizes that training and serving the layer give it:

  norm    the residual update and RMS norm before the layer; training runs its backward as well
  after   the weighted combine with the RMS norm after the layer, a gate and the scaled residual;
          training runs its backward as well
  ckpt    gate and up activations kept in 8 bits between a forward and its backward: codes and
          group scales, then g, u and h = SiLU(g) u restored from them
  gemm    products of int8 token rows with int8 expert weights, grouped by expert, a scale for each
          token and each channel; ffn: the SwiGLU expert FFN out of them, from bf16 token rows

With ``own`` false run() is the plain form (elementary torch operations in 32 bits); with ``own``
true it calls the library.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # one token of one request: launch latency alone
        dict(name="norm_decode_1", op="norm", T=1, H=2048, train=False, dtype="bf16"),
        # fp32 training of a small model, odd row count and width
        dict(name="norm_train_f32_1003", op="norm", T=1003, H=516, train=True, dtype="f32"),
        # the whole layer's training step, 16384 tokens
        dict(name="norm_train_16384", op="norm", T=16384, H=2048, train=True, dtype="bf16"),
        # a decode batch, gated element by element
        dict(name="after_decode_32", op="after", T=32, H=2048, E=128, k=8, gate="full", train=False,
             dtype="bf16"),
        # the whole layer's training step, a gate for each token
        dict(name="after_train_16384", op="after", T=16384, H=2048, E=128, k=8, gate="token",
             train=True, dtype="bf16"),
        # the tiny fp32 layer's gate and up, odd row count
        dict(name="ckpt_f32_517", op="ckpt", R=517, I=32, group=32, dtype="f32"),
        # the whole layer's gate and up: 16384 tokens, top-8
        dict(name="ckpt_full_131072", op="ckpt", R=131072, I=768, group=128, dtype="bf16"),
        # one product of ragged groups, one of them empty, odd widths
        dict(name="gemm_ragged_777", op="gemm", T=259, K=1040, N=528, E=5, k=3),
        # one token of one request through its eight experts
        dict(name="ffn_decode_1", op="ffn", T=1, H=2048, I=768, E=128, k=8, local=128),
        # a decode batch: nearly every expert has a few rows
        dict(name="ffn_decode_64", op="ffn", T=64, H=2048, I=768, E=128, k=8, local=128),
        # one expert-parallel rank's share of a prompt: 16 of 128 experts local
        dict(name="ffn_share_4096", op="ffn", T=4096, H=2048, I=768, E=128, k=8, local=16),
        # the whole 128-expert layer
        dict(name="ffn_full_16384", op="ffn", T=16384, H=2048, I=768, E=128, k=8, local=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "after", "ckpt", "gemm", "ffn", "ffn"])
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    if op == "norm":
        return dict(op=op, T=_log_int(rng, 1, 16384 if dtype == "bf16" else 8192),
                    H=8 * _log_int(rng, 8, 256), train=rng.random() < 0.6, dtype=dtype)
    if op == "after":
        E = rng.choice([8, 64, 128])
        return dict(op=op, T=_log_int(rng, 1, 16384 if dtype == "bf16" else 4096),
                    H=8 * _log_int(rng, 8, 256), E=E, k=rng.randint(2, 8),
                    gate=rng.choice(["none", "token", "full"]), train=rng.random() < 0.6, dtype=dtype)
    if op == "ckpt":
        group = rng.choice([32, 64, 128])
        return dict(op=op, R=_log_int(rng, 1, 131072 if dtype == "bf16" else 65536),
                    I=group * rng.randint(1, 768 // group), group=group, dtype=dtype)
    E = rng.choice([4, 8, 30, 64, 128])
    k = rng.randint(1, min(E, 8))
    if op == "gemm":
        return dict(op=op, T=_log_int(rng, 1, 16384), K=16 * _log_int(rng, 4, 128),
                    N=16 * _log_int(rng, 4, 96), E=E, k=k)
    return dict(op=op, T=_log_int(rng, 1, 16384), H=16 * _log_int(rng, 8, 128),
                I=16 * _log_int(rng, 4, 48), E=E, k=k, local=rng.choice([E, E // 2]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _routing(g, T, E, k, local):
    """Maps of a router that favours some experts: rows of one expert in token order, experts from
    `local` on elsewhere (dest -1).  Expert 1 of the small groups gets no token."""
    score = torch.rand((T, E), generator=g, device=DEV) + 0.3 * torch.rand((1, E), generator=g, device=DEV)
    if 1 < E <= 8 and k < E:
        score[:, 1] = -1.0
    idx = torch.topk(score, k, dim=1).indices.reshape(-1)
    key = torch.where(idx < local, idx, E)
    order = torch.argsort(key, stable=True)
    dest = torch.empty(T * k, dtype=torch.int64, device=DEV)
    dest[order] = torch.arange(T * k, device=DEV)
    dest = torch.where(idx < local, dest, -1)
    counts = torch.bincount(key, minlength=E + 1)[:local]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(counts, 0)])
    return dest.to(torch.int32), (order // k).to(torch.int32), offsets.to(torch.int32)


def _plan(offsets):
    """What a caller who knows the group sizes keeps for a padded product: the experts that have rows
    and the largest number of them."""
    counts = offsets[1:] - offsets[:-1]
    return dict(offsets=offsets, used=torch.nonzero(counts).squeeze(1), most=max(1, int(counts.max())))


def _weight_codes(g, E, N, K):
    """Codes and channel scales of weights of about unit gain."""
    q = (torch.randn((E, N, K), generator=g, device=DEV) * 36.0).round_().clamp_(-127, 127).to(torch.int8)
    return q, (torch.rand((E, N), generator=g, device=DEV) + 0.5) * (K ** -0.5 / 36.0)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    dt = TYPES[case.get("dtype", "bf16")]
    if op == "norm":
        T, H = case["T"], case["H"]
        s = dict(case=case, x=_normal(g, T, H, std=2.0, dtype=dt), delta=_normal(g, T, H, dtype=dt),
                 weight=1.0 + _normal(g, H, std=0.1), keep={})
        if case["train"]:
            s.update(dn=_normal(g, T, H, dtype=dt), dr=_normal(g, T, H, dtype=dt))
        return s
    if op == "after":
        T, H, E, k = (case[n] for n in ("T", "H", "E", "k"))
        dest, _, _ = _routing(g, T, E, k, E)
        s = dict(case=case, y_perm=_normal(g, T * k, H, std=0.5, dtype=dt), dest=dest,
                 w=torch.softmax(_normal(g, T, k), dim=1), residual=_normal(g, T, H, dtype=dt),
                 weight=1.0 + _normal(g, H, std=0.1), gate=None, keep={})
        if case["gate"] == "token":
            s["gate"] = torch.sigmoid(_normal(g, T))
        elif case["gate"] == "full":
            s["gate"] = torch.sigmoid(_normal(g, T, H)).to(dt)
        if case["train"]:
            s["dy"] = _normal(g, T, H, dtype=dt)
        return s
    if op == "ckpt":
        return dict(case=case, gu=_normal(g, case["R"], 2 * case["I"], dtype=dt), keep={})
    T, E, k = case["T"], case["E"], case["k"]
    if op == "gemm":
        K, N = case["K"], case["N"]
        _, src, offsets = _routing(g, T, E, k, E)
        q = (torch.randn((T, K), generator=g, device=DEV) * 36.0).round_().clamp_(-127, 127).to(torch.int8)
        w, ws = _weight_codes(g, E, N, K)
        return dict(case=case, x_q=q, x_scale=(torch.rand(T, generator=g, device=DEV) + 0.5) / 36.0,
                    src=src, offsets=offsets, w=w, w_scale=ws,
                    plan=_plan(offsets), keep={})
    H, I, local = case["H"], case["I"], case["local"]
    _, src, offsets = _routing(g, T, E, k, local)
    return dict(case=case, x=_normal(g, T, H, dtype=dt), src=src, offsets=offsets,
                plan=_plan(offsets), wg=_weight_codes(g, local, I, H),
                wu=_weight_codes(g, local, I, H), wd=_weight_codes(g, local, H, I),
                y_perm=torch.zeros((T * k, H), dtype=dt, device=DEV), keep={})


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "after": _own_after, "ckpt": _own_ckpt, "gemm": _own_gemm,
                "ffn": _own_ffn}[op](state)
    return {"norm": _plain_norm, "after": _plain_after, "ckpt": _plain_ckpt, "gemm": _plain_gemm,
            "ffn": _plain_ffn}[op](state)


# The library's calls.  state["keep"] holds the output buffers and workspaces that a training or
# serving loop keeps between its steps.

def _own_norm(s):
    import moe_expert_layer_router_amd as moe
    keep = s["keep"]
    f = moe.moe_norm(s["x"], s["weight"], EPS, delta=s["delta"], out=keep.get("fwd"))
    keep["fwd"] = f
    if not s["case"]["train"]:
        return dict(n=f["n"], r=f["r"])
    b = moe.moe_norm_bwd(s["dn"], f["r"], s["weight"], EPS, dr=s["dr"], ws=keep.get("ws"), out=keep.get("bwd"))
    keep.update(bwd=b, ws=b["ws"])
    return dict(n=f["n"], r=f["r"], dx=b["dx"], dweight=b["dweight"])


def _own_after(s):
    import moe_expert_layer_router_amd as moe
    keep = s["keep"]
    y = moe.moe_combine_norm(s["y_perm"], s["w"], s["dest"], s["case"]["T"], s["weight"], EPS,
                             residual=s["residual"], residual_scale=0.75, gate=s["gate"], out=keep.get("y"))
    keep["y"] = y
    if not s["case"]["train"]:
        return dict(y=y)
    b = moe.moe_combine_norm_bwd(s["dy"], s["y_perm"], s["w"], s["dest"], s["weight"], EPS, gate=s["gate"],
                                 ws=keep.get("ws"), out=keep.get("bwd"))
    keep.update(bwd=b, ws=b["ws"])
    got = dict(y=y, dy_perm=b["dy_perm"], d_topk_w=b["d_topk_w"], dweight=b["dweight"])
    if s["gate"] is not None:
        got["dgate"] = b["dgate"]
    return got


def _own_ckpt(s):
    import moe_expert_layer_router_amd as moe
    keep = s["keep"]
    q, scale = moe.moe_quantize_i8(s["gu"], group=s["case"]["group"], out=keep.get("codes"))
    r = moe.moe_swiglu_restore_i8(q, scale, s["gu"].dtype, out=keep.get("restored"))
    keep.update(codes={"q": q, "scale": scale}, restored=r)
    return dict(scale=scale, gu=r["gu"], h=r["h_perm"])


def _own_gemm(s):
    import moe_expert_layer_router_amd as moe
    s["keep"]["y"] = moe.moe_grouped_gemm_i8(s["x_q"], s["x_scale"], s["src"], s["offsets"], s["w"],
                                             s["w_scale"], out=s["keep"].get("y"))
    return dict(y=s["keep"]["y"])


def _own_ffn(s):
    import moe_expert_layer_router_amd as moe
    keep = s["keep"]
    q, scale = moe.moe_quantize_i8(s["x"], out=keep.get("codes"))
    f = moe.moe_grouped_ffn_fwd_i8(q, scale, s["src"], s["offsets"], s["wg"], s["wu"], s["wd"],
                                   ws=keep.get("ws"), out=keep.get("ffn") or {"y_perm": s["y_perm"]})
    keep.update(codes={"q": q, "scale": scale}, ffn=f, ws=f["ws"])
    return dict(y=f["y_perm"])


# The plain forms.

def _rms(v):
    return torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)


def _plain_norm(s):
    dt = s["x"].dtype
    r = (s["x"].float() + s["delta"].float()).to(dt)
    rf = r.float()
    rstd = _rms(rf)
    xh = rf * rstd
    n = (xh * s["weight"]).to(dt)
    if not s["case"]["train"]:
        return dict(n=n, r=r)
    dn = s["dn"].float()
    g = dn * s["weight"]
    dx = s["dr"].float() + rstd * (g - xh * (g * xh).mean(dim=1, keepdim=True))
    return dict(n=n, r=r, dx=dx.to(dt), dweight=(dn * xh).sum(dim=0))


def _plain_after(s):
    T, k, H = s["case"]["T"], s["case"]["k"], s["case"]["H"]
    dt, dest = s["y_perm"].dtype, s["dest"].long()
    rows = s["y_perm"][dest].float().reshape(T, k, H)
    c = (rows * s["w"].unsqueeze(2)).sum(dim=1)
    rstd = _rms(c)
    xh = c * rstd
    gate = 1.0
    if s["gate"] is not None:
        gate = s["gate"].float() if s["gate"].dim() == 2 else s["gate"].unsqueeze(1)
    y = (0.75 * s["residual"].float() + gate * (xh * s["weight"])).to(dt)
    if not s["case"]["train"]:
        return dict(y=y)
    dy = s["dy"].float()
    g = dy * gate * s["weight"]
    dc = rstd * (g - xh * (g * xh).mean(dim=1, keepdim=True))
    dy_perm = torch.empty_like(s["y_perm"])
    dy_perm[dest] = (dc.unsqueeze(1) * s["w"].unsqueeze(2)).to(dt).reshape(T * k, H)
    got = dict(y=y, dy_perm=dy_perm, d_topk_w=(rows * dc.unsqueeze(1)).sum(dim=2),
               dweight=(dy * gate * xh).sum(dim=0))
    if s["gate"] is not None:
        dgate = dy * (xh * s["weight"])
        got["dgate"] = dgate.to(dt) if s["gate"].dim() == 2 else dgate.sum(dim=1)
    return got


def _plain_codes(v, group):
    """Codes (as 32-bit values) and scales of the groups of `group` columns; whole-tensor divisors, so
    that both quotients are correctly rounded."""
    b = v.float().reshape(v.shape[0], -1, group)
    top = b.abs().amax(dim=2, keepdim=True)
    most = torch.full_like(top, 127.0)
    live = top >= 2.0 ** -100
    scale = torch.where(live, top / most, 0.0)
    q = torch.round(b * torch.where(live, most / torch.where(live, top, 1.0), 0.0))
    return q, scale


def _plain_ckpt(s):
    gu, I = s["gu"], s["case"]["I"]
    q, scale = _plain_codes(gu, s["case"]["group"])
    back = (q * scale).to(gu.dtype).reshape(gu.shape)
    gate, up = back[:, :I].float(), back[:, I:].float()
    return dict(scale=scale.squeeze(2), gu=back, h=(gate / (1.0 + torch.exp(-gate)) * up).to(gu.dtype))


def _plain_product(x, x_scale, plan, w, w_scale):
    """[R, N] products of the grouped rows x [R, K] (values of codes) in 32 bits: the rows of each expert
    that has some padded to the largest group, one batched product, the rows taken out again."""
    used, most, off = plan["used"], plan["most"], plan["offsets"].long()
    E, R, K, N = used.numel(), x.shape[0], x.shape[1], w.shape[1]
    row = torch.arange(R, device=x.device)
    e = torch.searchsorted(off[1:][used], row, right=True)
    at = e * most + row - off[used][e]
    pad = torch.zeros((E * most, K), device=x.device)
    pad[at] = x
    y = torch.bmm(pad.reshape(E, most, K), w[used].float().transpose(1, 2).contiguous())
    return y.reshape(E * most, N)[at] * x_scale.unsqueeze(1) * w_scale[used][e]


def _plain_gemm(s):
    src = s["src"].long()
    return dict(y=_plain_product(s["x_q"][src].float(), s["x_scale"][src], s["plan"], s["w"],
                                 s["w_scale"]).to(torch.bfloat16))


def _plain_ffn(s):
    plan, off = s["plan"], s["offsets"]
    q, scale = _plain_codes(s["x"], s["case"]["H"])
    live = torch.arange(s["src"].numel(), device=off.device) < off[-1]  # rows of the local experts
    src = s["src"].long()[live]
    x, xs = q.squeeze(1)[src], scale.reshape(-1)[src]
    g = _plain_product(x, xs, plan, *s["wg"])
    u = _plain_product(x, xs, plan, *s["wu"])
    h = (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16)
    hq, hs = _plain_codes(h, s["case"]["I"])
    s["y_perm"][live] = _plain_product(hq.squeeze(1), hs.reshape(-1), plan, *s["wd"]).to(torch.bfloat16)
    return dict(y=s["y_perm"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    e = 2 if case.get("dtype", "bf16") == "bf16" else 4
    if op == "norm":
        n = case["T"] * case["H"]
        return {"bytes": (8 if case["train"] else 4) * n * e + 4 * case["H"] * (3 if case["train"] else 1),
                "flops": (18 if case["train"] else 6) * n}
    if op == "after":
        T, H, k = case["T"], case["H"], case["k"]
        gate = {"none": 0, "token": T * 4, "full": T * H * e}[case["gate"]]
        b = T * k * H * e + 2 * T * H * e + T * k * 8 + H * 4 + gate
        f = 2 * T * k * H + 6 * T * H
        if case["train"]:
            b += 2 * T * k * H * e + T * H * e + T * k * 12 + 2 * H * 4 + 2 * gate
            f += 5 * T * k * H + 14 * T * H
        return {"bytes": b, "flops": f}
    if op == "ckpt":
        n = case["R"] * 2 * case["I"]
        return {"bytes": n * e + 2 * (n + 4 * n // case["group"]) + n * e + n * e // 2, "flops": 8 * n}
    T, E, k = case["T"], case["E"], case["k"]
    if op == "gemm":
        used = min(E, T * k)
        return {"bytes": T * (case["K"] + 4) + T * k * 4 + used * case["N"] * (case["K"] + 4)
                + T * k * case["N"] * 2, "flops": 2 * T * k * case["K"] * case["N"]}
    H, I, local = case["H"], case["I"], case["local"]
    rows = T * k * local / E
    used = min(local, local * (1.0 - (1.0 - k / E) ** T))  # experts that get a row
    return {"bytes": T * H * e + rows * 4 + used * (3 * H * I + 4 * (2 * I + H)) + rows * H * e,
            "flops": 6 * rows * H * I}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "after": _exact_after, "ckpt": _exact_ckpt, "gemm": _exact_gemm,
            "ffn": _exact_ffn}[case["op"]](s)


def _exact_norm(s):
    # r is the stored sum: what the norm and its backward read
    r = (s["x"].float() + s["delta"].float()).to(s["x"].dtype).double()
    w = s["weight"].double()
    inv = 1.0 / torch.sqrt(torch.mean(r ** 2, dim=1) + EPS)
    out = dict(n=r * inv[:, None] * w, r=r)
    if s["case"]["train"]:
        dn = s["dn"].double()
        dot = torch.sum(dn * w * r, dim=1)
        out["dx"] = s["dr"].double() + inv[:, None] * dn * w - r * (dot * inv ** 3 / r.shape[1])[:, None]
        out["dweight"] = torch.mv(torch.transpose(dn * r, 0, 1), inv)
    return out


def _exact_after(s):
    case = s["case"]
    T, k, H = case["T"], case["k"], case["H"]
    dest, w, weight = s["dest"].reshape(T, k).long(), s["w"].double(), s["weight"].double()
    c = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    for j in range(k):
        c += w[:, j, None] * s["y_perm"][dest[:, j]].double()
    inv = 1.0 / torch.sqrt(torch.mean(c ** 2, dim=1) + EPS)
    gate = torch.ones((T, 1), dtype=torch.float64, device=DEV)
    if s["gate"] is not None:
        gate = s["gate"].double().reshape(T, -1)
    z = c * inv[:, None]
    out = dict(y=0.75 * s["residual"].double() + gate * weight * z)
    if not case["train"]:
        return out
    dy = s["dy"].double()
    g = dy * gate * weight
    dc = inv[:, None] * g - c * (torch.sum(g * c, dim=1) * inv ** 3 / H)[:, None]
    dw = torch.zeros((T, k), dtype=torch.float64, device=DEV)
    dy_perm = torch.zeros((T * k, H), dtype=torch.float64, device=DEV)
    for j in range(k):
        dw[:, j] = torch.sum(dc * s["y_perm"][dest[:, j]].double(), dim=1)
        dy_perm[dest[:, j]] = w[:, j, None] * dc
    out.update(dy_perm=dy_perm, d_topk_w=dw, dweight=torch.sum(dy * gate * z, dim=0))
    if s["gate"] is not None:
        full = dy * weight * z
        out["dgate"] = full if s["gate"].dim() == 2 else torch.sum(full, dim=1)
    return out


def _exact_codes(v, group):
    """The codes that the definition gives in 32-bit arithmetic (numpy), as 64-bit values, and the scales."""
    b = v.float().cpu().numpy().reshape(v.shape[0], -1, group)
    top = np.abs(b).max(axis=2, keepdims=True).astype(np.float32)
    live = top >= np.float32(2.0 ** -100)
    inv = np.where(live, np.float32(127.0) / np.where(live, top, np.float32(1.0)), np.float32(0.0))
    scale = np.where(live, top / np.float32(127.0), np.float32(0.0))
    q = np.rint(b * inv.astype(np.float32))
    return (torch.from_numpy(q.reshape(v.shape)).to(DEV).double(),
            torch.from_numpy(scale[:, :, 0].astype(np.float32)).to(DEV).double())


def _exact_ckpt(s):
    gu, I, group = s["gu"], s["case"]["I"], s["case"]["group"]
    q, scale = _exact_codes(gu, group)
    back = q * torch.repeat_interleave(scale, group, dim=1)
    # h is formed from the restored values as they are stored
    kept = back.to(torch.float32).to(gu.dtype).double()
    return dict(scale=scale, gu=back, h=kept[:, :I] * torch.sigmoid(kept[:, :I]) * kept[:, I:])


def _exact_gemm(s):
    R, N = s["src"].numel(), s["case"]["N"]
    y = torch.zeros((R, N), dtype=torch.float64, device=DEV)
    off = s["offsets"].tolist()
    for e in range(len(off) - 1):
        src = s["src"][off[e]:off[e + 1]].long()
        p = s["x_q"][src].double() @ s["w"][e].double().t()
        y[off[e]:off[e + 1]] = s["x_scale"][src].double()[:, None] * p * s["w_scale"][e].double()
    return dict(y=y)


def _exact_ffn(s):
    q, scale = _exact_codes(s["x"], s["case"]["H"])
    y = torch.zeros(s["y_perm"].shape, dtype=torch.float64, device=DEV)
    off = s["offsets"].tolist()
    for e in range(len(off) - 1):
        if off[e] == off[e + 1]:
            continue
        src = s["src"][off[e]:off[e + 1]].long()
        xs = scale[src]
        g = xs * (q[src] @ s["wg"][0][e].double().t()) * s["wg"][1][e].double()
        u = xs * (q[src] @ s["wu"][0][e].double().t()) * s["wu"][1][e].double()
        # h is quantized as it is stored, in bf16
        h = (g * torch.sigmoid(g) * u).to(torch.float32).to(torch.bfloat16)
        hq, hs = _exact_codes(h, s["case"]["I"])
        y[off[e]:off[e + 1]] = hs * (hq @ s["wd"][0][e].double().t()) * s["wd"][1][e].double()
    return dict(y=y)
