"""What the operators around the MoE expert layer cost.

Three operators, each on the sizes that training, fine-tuning and serving the
layer give it:

  balance   load-balance and z loss of a router's logits with the per-expert
            counts, and the gradient of the logits (one training step: forward
            and backward)
  dropout   the weighted combine with dropout from a counter-based generator
            and the residual added, and its backward (one training step)
  adapter   low-rank adapters of many requests added to a projection's output;
            serving runs the forward alone, training the backward as well

With ``own`` false run() is the plain form (elementary torch operations in 32
bits); with ``own`` true it calls the library.
"""
import functools
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the tiny fp32 layer's router over three ragged sequences, one empty:
        # the smallest step, launch latency alone
        dict(name="balance_tiny_256", op="balance", T=256, E=8, k=2, S=3, mask=0.0),
        # an expert-parallel rank's training step: 8192 tokens, 128 experts, top-8
        dict(name="balance_train_8192", op="balance", T=8192, E=128, k=8, S=1, mask=0.0),
        # packed sequences of different lengths with padding masked out
        dict(name="balance_packed_32768", op="balance", T=32768, E=128, k=8, S=24, mask=0.1),
        # the tiny fp32 layer's combine
        dict(name="dropout_tiny_f32_256", op="dropout", T=256, H=64, E=8, k=2, lo=0, hi=8, p=0.1,
             dtype="f32"),
        # one expert-parallel rank's share: 16 of 128 experts local, about one
        # local slot for each token
        dict(name="dropout_share_8192", op="dropout", T=8192, H=2048, E=128, k=8, lo=0, hi=16, p=0.1,
             dtype="bf16"),
        # the whole 128-expert layer
        dict(name="dropout_full_16384", op="dropout", T=16384, H=2048, E=128, k=8, lo=0, hi=128,
             p=0.05, dtype="bf16"),
        # one token of one request
        dict(name="adapter_decode_1", op="adapter", R=1, K=2048, N=2048, ids=32, rank=16,
             order="mixed", gather=False, train=False, dtype="bf16"),
        # a decode batch whose requests use 64 adapters
        dict(name="adapter_decode_128", op="adapter", R=128, K=2048, N=2048, ids=64, rank=16,
             order="mixed", gather=False, train=False, dtype="bf16"),
        # prompts of eight requests packed one after another, rank 64
        dict(name="adapter_prompts_8191", op="adapter", R=8191, K=2048, N=1536, ids=8, rank=64,
             order="sorted", gather=False, train=False, dtype="bf16"),
        # fp32 fine-tuning of a small projection, odd row count, mixed rows
        dict(name="adapter_train_f32_1003", op="adapter", R=1003, K=516, N=260, ids=5, rank=8,
             order="mixed", gather=False, train=True, dtype="f32"),
        # a rank's down projection while training: 16 local experts, one
        # adapter for each, rows grouped by expert
        dict(name="adapter_train_share_8285", op="adapter", R=8285, K=768, N=2048, ids=16, rank=16,
             order="sorted", gather=False, train=True, dtype="bf16"),
        # the whole layer's gate and up projection: 16384 tokens, top-8, 128
        # experts, token rows read through the permutation
        dict(name="adapter_train_full_131072", op="adapter", R=131072, K=2048, N=1536, ids=128,
             rank=16, order="sorted", gather=True, train=True, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "dropout", "adapter", "adapter"])
    if op == "balance":
        T = _log_int(rng, 64, 32768)
        E = rng.randint(4, 256) if rng.random() < 0.5 else rng.choice([8, 16, 64, 128])
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 8)), S=_log_int(rng, 1, min(T, 64)),
                    mask=rng.choice([0.0, 0.1, 0.5]))
    if op == "dropout":
        E = rng.choice([8, 64, 128])
        T, H = _log_int(rng, 16, 16384), 8 * _log_int(rng, 8, 256)
        lo = rng.choice([0, E // 2])
        return dict(op=op, T=T, H=H, E=E, k=rng.randint(1, 8), lo=lo, hi=rng.choice([lo + E // 4, E]),
                    p=round(rng.uniform(0.01, 0.5), 3),
                    dtype="bf16" if rng.random() < 0.7 or T * H > 1 << 24 else "f32")
    dtype = "bf16" if rng.random() < 0.75 else "f32"
    train = rng.random() < 0.5
    R = _log_int(rng, 64 if train else 1, 32768 if dtype == "bf16" else 8192)
    return dict(op=op, R=R, K=8 * _log_int(rng, 8, 256), N=8 * _log_int(rng, 8, 256),
                ids=_log_int(rng, 1, 128), rank=rng.choice([8, 16, 24, 32, 64]),
                order=rng.choice(["sorted", "mixed"]), gather=rng.random() < 0.3, train=train,
                dtype=dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _lengths(seed, T, S):
    """Offsets of S sequences that fill T rows; the second of three or more is empty."""
    r = np.random.RandomState(seed % (1 << 31))
    cuts = np.sort(r.randint(0, T + 1, S - 1))
    if S >= 3:
        cuts[1] = cuts[0]
    return np.concatenate([[0], cuts, [T]]).astype(np.int32)


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        # a trained router's logits: unit normals, some experts favoured
        logits = _normal(g, T, E) + _normal(g, 1, E)
        idx = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
        mask = None
        if case["mask"] > 0:
            mask = (torch.rand(T, generator=g, device=DEV) >= case["mask"]).to(torch.uint8)
        offsets = torch.from_numpy(_lengths(seed, T, S)).to(DEV)
        return dict(case=case, logits=logits, idx=idx, mask=mask, offsets=offsets,
                    coef=(0.01, 0.001), d_loss=_normal(g, 1).abs() + 0.5, keep={})
    dt = TYPES[case["dtype"]]
    if case["op"] == "dropout":
        T, H, E, k, lo, hi = (case[n] for n in ("T", "H", "E", "k", "lo", "hi"))
        # routing of a favoured-expert router, rows of one expert in token order
        score = torch.rand((T, E), generator=g, device=DEV)
        idx = torch.topk(score, k, dim=1).indices.reshape(-1)
        local = (idx >= lo) & (idx < hi)
        order = torch.argsort(torch.where(local, idx, E), stable=True)
        dest = torch.empty(T * k, dtype=torch.int32, device=DEV)
        dest[order] = torch.arange(T * k, dtype=torch.int32, device=DEV)
        dest = torch.where(local, dest, -1).contiguous()
        w = torch.softmax(_normal(g, T, k), dim=1)
        rows = torch.arange(T * k, device=DEV).unsqueeze(1) < local.sum()
        y_perm = _normal(g, T * k, H, std=0.5, dtype=dt) * rows
        return dict(case=case, y_perm=y_perm, w=w, dest=dest, residual=_normal(g, T, H, dtype=dt),
                    dy=_normal(g, T, H, dtype=dt), p=case["p"],
                    rng=torch.tensor([int(seed) * 2654435761 % (1 << 62), int(seed) % 1000],
                                     dtype=torch.int64, device=DEV),
                    dy_perm=torch.zeros((T * k, H), dtype=dt, device=DEV), keep={})
    R, K, N, ids, rank = (case[n] for n in ("R", "K", "N", "ids", "rank"))
    row_id = torch.randint(0, ids, (R,), generator=g, device=DEV, dtype=torch.int32)
    if R >= 16:  # requests without an adapter
        row_id[torch.rand(R, generator=g, device=DEV) < 0.03] = -1
    if case["order"] == "sorted":
        row_id = torch.sort(row_id).values.contiguous()
    rows = max(1, R // 8) if case["gather"] else R
    src = None
    if case["gather"]:
        src = torch.randint(0, rows, (R,), generator=g, device=DEV, dtype=torch.int32)
    s = dict(case=case, row_id=row_id, src=src, x=_normal(g, rows, K, dtype=dt),
             A=_normal(g, ids, rank, K, std=K ** -0.5, dtype=dt),
             B=_normal(g, ids, N, rank, std=rank ** -0.5, dtype=dt),
             scale=torch.rand(ids, generator=g, device=DEV) + 0.5, y=_normal(g, R, N, dtype=dt), keep={})
    if case["train"]:
        s["dy"] = _normal(g, R, N, dtype=dt)
        s["dx"] = _normal(g, R, K, dtype=dt)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if op == "balance":
        return _own_balance(state) if own else _plain_balance(state)
    if op == "dropout":
        return _own_dropout(state) if own else _plain_dropout(state)
    return _own_adapter(state) if own else _plain_adapter(state)


# The library's calls.  state["keep"] holds the output buffers and workspaces
# that a training or serving loop keeps between its steps.

def _own_balance(s):
    import moe_expert_layer_router_amd as moe
    k, (cb, cz) = s["case"]["k"], s["coef"]
    f = moe.moe_balance_loss(s["logits"], s["idx"], cb, cz, seq_offsets=s["offsets"],
                             token_mask=s["mask"], ws=s["keep"].get("ws"), out=s["keep"].get("fwd"))
    d = moe.moe_balance_loss_bwd(s["logits"], f, k, cb, cz, d_loss=s["d_loss"],
                                 seq_offsets=s["offsets"], token_mask=s["mask"],
                                 out=s["keep"].get("d_logits"))
    s["keep"].update(fwd=f, d_logits=d, ws=f["ws"])
    return dict(loss=f["loss"], counts=f["counts"], prob_sum=f["prob_sum"], d_logits=d)


def _own_dropout(s):
    import moe_expert_layer_router_amd as moe
    y = moe.moe_combine_dropout(s["y_perm"], s["w"], s["dest"], s["case"]["T"], s["p"], s["rng"],
                                residual=s["residual"], out=s["keep"].get("y"))
    b = moe.moe_combine_dropout_bwd(s["dy"], s["y_perm"], s["w"], s["dest"], s["p"], s["rng"],
                                    out=s["keep"].get("bwd") or {"dy_perm": s["dy_perm"]})
    s["keep"].update(y=y, bwd=b)
    return dict(y=y, dy_perm=b["dy_perm"], d_topk_w=b["d_topk_w"])


def _own_adapter(s):
    import moe_expert_layer_router_amd as moe
    train = s["case"]["train"]
    v = moe.moe_adapter_fwd(s["x"], s["row_id"], s["A"], s["B"], s["y"], scale=s["scale"],
                            src_row=s["src"], want_v=train, out=s["keep"].get("v"))
    if not train:
        return dict(y=s["y"])
    b = moe.moe_adapter_bwd(s["dy"], s["x"], s["row_id"], s["A"], s["B"], v, s["dx"],
                            scale=s["scale"], src_row=s["src"], ws=s["keep"].get("ws"),
                            out=s["keep"].get("bwd"))
    s["keep"].update(v=v, bwd=b, ws=b["ws"])
    return dict(y=s["y"], dx=s["dx"], dA=b["dA"], dB=b["dB"])


# The plain forms.

def _plain_balance(s):
    z, idx, off, (cb, cz) = s["logits"], s["idx"], s["offsets"], s["coef"]
    T, E = z.shape
    k, S = s["case"]["k"], off.numel() - 1
    live = torch.ones(T, device=z.device) if s["mask"] is None else s["mask"].float()
    t = torch.arange(T, device=z.device)
    member = ((t >= off[:-1, None]) & (t < off[1:, None])).float() * live  # [S, T]
    top = z.max(dim=1, keepdim=True).values
    ex = torch.exp(z - top)
    total = ex.sum(dim=1, keepdim=True)
    p = ex / total
    lse = (top + torch.log(total)).squeeze(1)
    picked = (idx.unsqueeze(2) == torch.arange(E, device=z.device)).sum(dim=1).float()  # [T, E]
    c, q = member @ picked, member @ p
    n = member.sum(dim=1)
    rows = n.sum().clamp(min=1.0)
    per = E / (k * rows * n.clamp(min=1.0))  # [S]
    balance = (per * (c * q).sum(dim=1)).sum()
    zl = (member.sum(dim=0) * lse * lse).sum() / rows
    mine = member.t() @ (per[:, None] * c)  # [T, E]: each row's sequence
    d = s["d_loss"] * p * (cb * (mine - (p * mine).sum(dim=1, keepdim=True))
                           + (cz * 2.0 / rows) * (lse * member.sum(dim=0))[:, None])
    return dict(loss=torch.stack([balance, zl, cb * balance + cz * zl]), counts=c.to(torch.int32),
                prob_sum=q, d_logits=d)


def _philox_round(c, key):
    """One round of Philox4x32 on int64 tensors that hold 32-bit words."""
    low = 0xFFFFFFFF
    p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
    return [((p1 >> 32) & low) ^ c[1] ^ key[0], p1 & low, ((p0 >> 32) & low) ^ c[3] ^ key[1], p0 & low]


def _keep_mask(rng, T, H, p):
    """keep[t, h]: word i % 4 of Philox4x32-10 at counter (i // 4, offset), i = t H + h, is at
    least floor(p 2^32)."""
    low = 0xFFFFFFFF
    seed, offset = rng[0], rng[1]
    i = torch.arange(T * H // 4, device=rng.device)
    key = [seed & low, (seed >> 32) & low]
    start = [i & low, i >> 32, (offset & low).expand_as(i), ((offset >> 32) & low).expand_as(i)]
    words = functools.reduce(
        lambda c, n: _philox_round(c, [(key[0] + n * 0x9E3779B9) & low, (key[1] + n * 0xBB67AE85) & low]),
        range(10), start)
    return (torch.stack(words, dim=1) >= int(p * 4294967296.0)).reshape(T, H)


def _plain_dropout(s):
    T, H = s["residual"].shape
    k = s["w"].shape[1]
    keep = _keep_mask(s["rng"], T, H, s["p"]).float() / (1.0 - s["p"])
    local = (s["dest"] >= 0).reshape(T, k)
    rows = s["y_perm"][s["dest"].clamp(min=0).long()].float().reshape(T, k, H)
    w = torch.where(local, s["w"], 0.0)
    y = (s["residual"].float() + keep * (rows * w.unsqueeze(2)).sum(dim=1)).to(s["residual"].dtype)
    g = s["dy"].float() * keep
    dw = torch.where(local, (rows * g.unsqueeze(1)).sum(dim=2), 0.0)
    d = (g.unsqueeze(1) * w.unsqueeze(2)).to(s["dy"].dtype).reshape(T * k, H)
    s["dy_perm"][s["dest"][local.reshape(-1)].long()] = d[local.reshape(-1)]
    return dict(y=y, dy_perm=s["dy_perm"], d_topk_w=dw)


def _plain_adapter(s):
    ids, rank, K = s["A"].shape
    x = (s["x"] if s["src"] is None else s["x"][s["src"].long()]).float()
    A = s["A"].float().reshape(ids * rank, K)
    B = s["B"].float().transpose(1, 2).reshape(ids * rank, -1)
    # every adapter's product, then each row keeps its own adapter's columns
    mine = (s["row_id"].unsqueeze(1) == torch.arange(ids, device=x.device)).float() * s["scale"]
    mine = mine.repeat_interleave(rank, dim=1)
    v = (x @ A.t()) * mine
    s["y"].copy_(s["y"].float() + v @ B)
    if not s["case"]["train"]:
        return dict(y=s["y"])
    dy = s["dy"].float()
    dv = (dy @ B.t()) * mine
    s["dx"].copy_(s["dx"].float() + dv @ A)
    dA = (dv.t() @ x).reshape(ids, rank, K)
    dB = (v.t() @ dy).reshape(ids, rank, -1).transpose(1, 2).contiguous()
    return dict(y=s["y"], dx=s["dx"], dA=dA, dB=dB)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        # forward: logits and choices in, counts and sums out; backward: logits
        # in, their gradient out
        b = T * E * 4 + T * k * 4 + T * (1 if case["mask"] else 0) + 2 * case["S"] * E * 4 + 2 * T * E * 4
        return {"bytes": b, "flops": 12 * T * E}
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "dropout":
        T, H, k = case["T"], case["H"], case["k"]
        slots = T * k * (case["hi"] - case["lo"]) / case["E"]
        maps = T * k * 8
        fwd = slots * H * e + 2 * T * H * e + maps
        bwd = T * H * e + 2 * slots * H * e + maps + T * k * 4
        return {"bytes": fwd + bwd, "flops": 2 * slots * H + 4 * slots * H + 2 * T * H}
    R, K, N, ids, rank = (case[n] for n in ("R", "K", "N", "ids", "rank"))
    used = min(ids, R)
    rows = max(1, R // 8) if case["gather"] else R
    weights = used * rank * (K + N) * e
    b = rows * K * e + 2 * R * N * e + weights + R * 4
    f = 2 * R * rank * (K + N)
    if case["train"]:
        b += R * N * e + rows * K * e + 2 * R * K * e + weights + ids * rank * (K + N) * 4 + R * 4
        f += 4 * R * rank * (K + N)
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"balance": _exact_balance, "dropout": _exact_dropout, "adapter": _exact_adapter}[case["op"]](s)


def _exact_balance(s):
    z = s["logits"].cpu().numpy().astype(np.float64)
    idx, off = s["idx"].cpu().numpy(), s["offsets"].cpu().numpy()
    T, E = z.shape
    k, S, (cb, cz) = s["case"]["k"], len(off) - 1, s["coef"]
    live = np.ones(T, bool) if s["mask"] is None else s["mask"].cpu().numpy() != 0
    N = sum(int(live[off[i]:off[i + 1]].sum()) for i in range(S))
    counts, q, d = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros((T, E))
    balance = zl = 0.0
    g = float(s["d_loss"].item())
    for i in range(S):
        at = np.arange(off[i], off[i + 1])[live[off[i]:off[i + 1]]]
        n = len(at)
        if n == 0:
            continue
        zs = z[at]
        lse = np.logaddexp.reduce(zs, axis=1)
        p = np.exp(zs - lse[:, None])
        counts[i] = np.bincount(idx[at].reshape(-1), minlength=E)
        q[i] = p.sum(axis=0)
        f = E * counts[i] / (k * n)
        balance += n / N * float(f @ (q[i] / n))
        zl += float((lse ** 2).sum()) / N
        d[at] = g * p * (cb / N * (f - p @ f[:, None]) + cz * 2.0 / N * lse[:, None])
    return dict(loss=np.array([balance, zl, cb * balance + cz * zl]), counts=counts.astype(np.int32),
                prob_sum=q, d_logits=d)


def _philox_words(seed, offset, n):
    """The words of Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011) at counters 0 .. n-1."""
    u, low = np.uint64, np.uint64(0xFFFFFFFF)
    i = np.arange(n, dtype=np.uint64)
    c0, c1 = i & low, i >> u(32)
    c2, c3 = np.full(n, offset & 0xFFFFFFFF, u), np.full(n, offset >> 32, u)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c0 * u(0xD2511F53), c2 * u(0xCD9E8D57)
        c0, c1, c2, c3 = (b >> u(32)) ^ c1 ^ u(k0), b & low, (a >> u(32)) ^ c3 ^ u(k1), a & low
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack([c0, c1, c2, c3], axis=1).reshape(-1)


def _exact_dropout(s):
    case = s["case"]
    T, H, k, p = case["T"], case["H"], case["k"], case["p"]
    seed, offset = (int(v) for v in s["rng"].cpu())
    keep = torch.from_numpy(_philox_words(seed, offset, T * H // 4) >= np.uint64(int(p * 2 ** 32)))
    keep = keep.to(DEV).reshape(T, H).double() / (1.0 - p)
    dest = s["dest"].reshape(T, k).long()
    w = s["w"].double()
    y = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    dw = torch.zeros((T, k), dtype=torch.float64, device=DEV)
    dy_perm = torch.zeros_like(s["dy_perm"], dtype=torch.float64)
    g = s["dy"].double() * keep
    for j in range(k):
        t = torch.nonzero(dest[:, j] >= 0).squeeze(1)
        r = dest[t, j]
        rows = s["y_perm"][r].double()
        y[t] += w[t, j, None] * rows
        dw[t, j] = (rows * g[t]).sum(dim=1)
        dy_perm[r] = w[t, j, None] * g[t]
    return dict(y=s["residual"].double() + keep * y, dy_perm=dy_perm, d_topk_w=dw)


def _exact_adapter(s):
    case = s["case"]
    x, A, B = s["x"].double(), s["A"].double(), s["B"].double()
    scale = s["scale"].double()
    y = s["y"].double()
    out = dict(y=y)
    if case["train"]:
        dy, dx = s["dy"].double(), s["dx"].double()
        out.update(dx=dx, dA=torch.zeros_like(A), dB=torch.zeros_like(B))
    for a in range(case["ids"]):
        r = torch.nonzero(s["row_id"] == a).squeeze(1)
        if r.numel() == 0:
            continue
        xr = x[r] if s["src"] is None else x[s["src"][r].long()]
        v = scale[a] * (xr @ A[a].t())
        y[r] += v @ B[a].t()
        if case["train"]:
            dv = scale[a] * (dy[r] @ B[a])
            dx[r] += dv @ A[a]
            out["dA"][a] = dv.t() @ xr
            out["dB"][a] = dy[r].t() @ v
    return out
