"""Auxiliary losses of the router (moe_balance_loss, its gradient, moe_route_bwd_add)
against float64 definitions.

Tolerances (u = 2^-24, half an fp32 step relative to a value):
  lse       |d| <= (2 |lse| + E + 16) u: top and log rounded, E terms summed
  p         relative (128 + E + 8) u: the exponent's argument is off by u |z - top| with
            |z - top| < 104 wherever p is not 0, E terms summed, a division; p below the
            normal range may lose everything: 2^-126 absolute
  prob_sum  relative (n + 128 + E + 8) u for n summed rows of positive terms
  loss      relative (n + 2 (128 + E + 8)) u + the lse bound twice
  d_logits  g p (kb (c + sum p c) + kz |lse|) times 4 (128 + E + 16) u
"""
import ctypes

import numpy as np
import pytest
import torch

from test_abi_cpu import A, EINVAL, EWS, F32, BF16, L, N, OK, S as STREAM, U, _err
import moe_expert_layer_router_amd as moe

DEV = torch.device("cuda:0")
U24 = 2.0 ** -24
gpu = pytest.mark.gpu


def softmax_rows(z):
    """(p, lse) in 64 bits; a row of -inf alone has p = 0 and lse = 0."""
    top = z.max(axis=1, keepdims=True)
    none = np.isneginf(top)
    ex = np.where(none, 0.0, np.exp(z - np.where(none, 0.0, top)))
    total = ex.sum(axis=1, keepdims=True)
    p = ex / np.where(none, 1.0, total)
    lse = np.where(none, 0.0, np.where(none, 0.0, top) + np.log(np.where(none, 1.0, total)))
    return p, lse[:, 0]


def reference(z, idx, k, off, live, cb, cz, g=1.0, counts=None):
    T, E = z.shape
    S = len(off) - 1
    live = live & (np.arange(T) >= off[0]) & (np.arange(T) < off[-1])
    p, lse = softmax_rows(np.where(live[:, None], z.astype(np.float64), 0.0))
    p[~live], lse[~live] = 0.0, 0.0
    n = np.array([live[off[s]:off[s + 1]].sum() for s in range(S)])
    N_all = n.sum()
    c, q, d = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros((T, E))
    mag = np.zeros((T, E))
    bal = 0.0
    for s in range(S):
        rows = np.arange(off[s], off[s + 1])[live[off[s]:off[s + 1]]]
        if len(rows) == 0:
            continue
        picks = idx[rows].reshape(-1)
        c[s] = np.bincount(picks[(picks >= 0) & (picks < E)], minlength=E)
        if counts is not None:
            c[s] = counts[s]
        q[s] = p[rows].sum(axis=0)
        bal += E / (k * N_all * n[s]) * (c[s] * q[s]).sum()
        kb, kz = cb * E / (k * N_all * n[s]), 2 * cz * lse[rows] / N_all
        pc = p[rows] @ c[s]
        d[rows] = g * p[rows] * (kb * (c[s] - pc[:, None]) + kz[:, None])
        mag[rows] = abs(g) * p[rows] * (abs(kb) * (c[s] + pc[:, None]) + np.abs(kz)[:, None])
    zl = (lse ** 2).sum() / N_all if N_all else 0.0
    return dict(loss=np.array([bal, zl, cb * bal + cz * zl]), counts=c, prob_sum=q, lse=lse,
                tokens=np.append(n, N_all), d_logits=d, mag=mag)


def test_formula_gradient_matches_differences():
    rng = np.random.default_rng(0)
    T, E, k = 23, 6, 2
    off, live = np.array([2, 9, 9, 21]), rng.random(T) > 0.2
    z = rng.standard_normal((T, E))
    idx = np.argsort(-z, axis=1)[:, :k]
    ref = reference(z, idx, k, off, live, 0.7, 0.3)
    for t in range(T):
        for e in range(E):
            h = np.zeros((T, E))
            h[t, e] = 1e-6
            num = [reference(z + sign * h, idx, k, off, live, 0.7, 0.3, counts=ref["counts"])["loss"][2]
                   for sign in (1, -1)]
            # central differences of a smooth function: about h^2 + 2^-52 / h
            assert abs((num[0] - num[1]) / 2e-6 - ref["d_logits"][t, e]) < 1e-8


def test_even_routing_has_loss_one():
    E, k = 8, 2
    z = np.zeros((16, E))
    idx = np.stack([np.arange(16) % E, (np.arange(16) + 3) % E], axis=1)
    loss = reference(z, idx, k, np.array([0, 16]), np.ones(16, bool), 1.0, 0.0)["loss"]
    assert abs(loss[0] - 1.0) < 1e-12


def test_refusals():
    f = L.moe_balance_loss
    big = 1 << 30
    ok = [A, A, N, N, 32, 8, 2, 1, 0.1, 0.1, A, A, A, A, A, A, big, STREAM]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(_4=-1) == EINVAL
    assert call(_4=2 ** 26 - 1, _5=64, _6=32) == -2 and "T * k" in _err()
    assert call(_4=2 ** 31 - 1, _5=1, _6=1) == -2 and L.moe_balance_ws_bytes(2 ** 31 - 1, 1, 1) == -2
    assert call(_5=257) == EINVAL and call(_5=0) == EINVAL
    assert call(_6=0) == EINVAL and call(_6=9) == EINVAL
    assert call(_7=0) == EINVAL
    assert call(_7=3) == EINVAL and "seq_offsets" in _err()
    for i, name in ((0, "logits"), (1, "topk_idx"), (10, "counts"), (11, "prob_sum"), (12, "tokens"),
                    (13, "lse"), (14, "loss")):
        assert call(**{f"_{i}": N}) == EINVAL and name in _err()
    assert call(_15=N) == EWS and call(_16=16) == EWS
    assert call(_15=U) == EINVAL and "aligned" in _err()
    assert L.moe_balance_ws_bytes(-1, 8, 1) == EINVAL
    assert L.moe_balance_ws_bytes(8, 300, 1) == EINVAL
    assert L.moe_balance_ws_bytes(8, 8, 0) == EINVAL
    assert L.moe_balance_ws_bytes(0, 8, 1) > 0
    g = L.moe_balance_loss_bwd
    assert g(N, A, A, A, N, N, N, 32, 8, 2, 1, 0.1, 0.1, 0, A, STREAM) == EINVAL and "logits" in _err()
    assert g(A, A, A, A, N, N, N, 32, 8, 2, 1, 0.1, 0.1, 2, A, STREAM) == EINVAL and "accumulate" in _err()
    assert g(A, A, A, A, N, N, N, 32, 8, 2, 1, 0.1, 0.1, 0, N, STREAM) == EINVAL and "d_logits" in _err()
    assert g(A, A, A, A, N, N, N, 32, 8, 2, 4, 0.1, 0.1, 0, A, STREAM) == EINVAL
    assert g(A, A, A, A, N, N, N, 0, 8, 2, 1, 0.1, 0.1, 0, A, STREAM) == OK
    r = L.moe_route_bwd_add
    assert r(A, A, A, N, A, A, 32, 64, 8, 2, F32, A, N, N, A, big, STREAM) == EINVAL and "d_logits_add" in _err()
    assert r(A, A, A, A, A, A, 32, 96, 8, 2, BF16, A, N, N, A, big, STREAM) == -2
    assert r(A, A, A, A, A, A, 32, 64, 8, 2, F32, N, N, N, A, big, STREAM) == EINVAL and "d_logits" in _err()


def test_binding_refuses_cpu_tensors():
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_balance_loss(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), 0.1)


# ---------------------------------------------------------------------------
# on the GPU
# ---------------------------------------------------------------------------

def offsets_of(rng, T, S):
    cuts = np.sort(rng.integers(0, T + 1, S - 1))
    if S >= 3:
        cuts[1] = cuts[0]  # an empty sequence
    return np.concatenate([[0], cuts, [T]]).astype(np.int32)


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV) if dtype is None else \
        torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def compare(got, d_logits, ref, E):
    n = max(1, ref["tokens"][-1])
    perr = (128 + E + 8) * U24
    lerr = (2 * np.abs(ref["lse"]) + E + 16) * U24
    host = {k: got[k].cpu().numpy() for k in ("loss", "counts", "prob_sum", "lse", "tokens")}
    assert np.array_equal(host["counts"], ref["counts"])
    assert np.array_equal(host["tokens"], ref["tokens"])
    assert (np.abs(host["lse"] - ref["lse"]) <= lerr).all()
    assert (np.abs(host["prob_sum"] - ref["prob_sum"])
            <= (n * U24 + perr) * ref["prob_sum"] + n * 2.0 ** -126).all()
    zmag = 2 * (np.abs(ref["lse"]) * lerr).sum() / n
    lim = (n * U24 + 2 * perr) * np.abs(ref["loss"]) + np.array([1e-37, zmag, zmag])
    assert (np.abs(host["loss"] - ref["loss"]) <= lim).all(), (host["loss"], ref["loss"])
    if d_logits is not None:
        err = np.abs(d_logits.cpu().numpy() - ref["d_logits"])
        assert (err <= 4 * (perr + 8 * U24) * ref["mag"] + 2.0 ** -126).all(), err.max()


CASES = [  # T, E, k, S, mask
    (1, 1, 1, 1, 0.0), (1, 8, 2, 1, 0.0), (2, 256, 32, 2, 0.0), (33, 5, 3, 4, 0.3), (64, 8, 2, 1, 0.0),
    (257, 60, 4, 5, 0.1), (300, 33, 7, 300, 0.2), (1000, 64, 6, 3, 0.5), (4097, 128, 8, 7, 0.1),
    (5000, 129, 1, 1, 0.0), (20000, 254, 8, 40, 0.1), (100, 130, 2, 5000, 0.0),
]


@gpu
@pytest.mark.parametrize("T,E,k,S,drop", CASES)
def test_against_definition(T, E, k, S, drop):
    rng = np.random.default_rng(T * 1000 + E)
    z = (rng.standard_normal((T, E)) * 2 + rng.standard_normal(E)).astype(np.float32)
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    off = offsets_of(rng, T, S) if S > 1 else np.array([0, T], np.int32)
    live = rng.random(T) >= drop
    ref = reference(z, idx, k, off, live, 0.02, 0.003, g=1.7)
    zd, id_, md = dev(z), dev(idx), dev(live.astype(np.uint8)) if drop else None
    od = dev(off) if S > 1 else None
    f = moe.moe_balance_loss(zd, id_, 0.02, 0.003, seq_offsets=od, token_mask=md)
    g = torch.tensor([1.7], device=DEV)
    d = moe.moe_balance_loss_bwd(zd, f, k, 0.02, 0.003, d_loss=g, seq_offsets=od, token_mask=md)
    ref = reference(z, idx, k, off, live, np.float32(0.02), np.float32(0.003), g=np.float32(1.7))
    compare(f, d, ref, E)
    # the same bits again, and an accumulating gradient
    f2 = moe.moe_balance_loss(zd, id_, 0.02, 0.003, seq_offsets=od, token_mask=md)
    for n in ("loss", "prob_sum", "lse"):
        assert torch.equal(f[n].view(torch.int32), f2[n].view(torch.int32))
    base = torch.full_like(d, 0.25)
    moe.moe_balance_loss_bwd(zd, f, k, 0.02, 0.003, d_loss=g, seq_offsets=od, token_mask=md,
                             accumulate=True, out=base)
    assert torch.equal(base, d + 0.25)


@gpu
def test_rows_outside_the_sequences_and_masked_rows_do_not_count():
    """Gap before the first sequence, rows behind the last, masked rows of NaN and inf."""
    rng = np.random.default_rng(5)
    T, E, k = 100, 12, 2
    z = rng.standard_normal((T, E)).astype(np.float32)
    idx = np.argsort(-z, axis=1)[:, :k].astype(np.int32)
    off, live = np.array([7, 40, 40, 81], np.int32), rng.random(T) > 0.4
    ref = reference(z, idx, k, off, live, 0.5, 0.25)
    bad = np.array([np.nan, np.inf, -np.inf], np.float32)
    junk = ~live | (np.arange(T) < 7) | (np.arange(T) >= 81)
    z[junk] = bad[rng.integers(0, 3, (junk.sum(), E))]
    idx[junk] = rng.choice([-5, 3, 1 << 30], (junk.sum(), k))
    f = moe.moe_balance_loss(dev(z), dev(idx), 0.5, 0.25, seq_offsets=dev(off),
                             token_mask=dev(live.astype(np.uint8)))
    d = torch.full((T, E), float("nan"), device=DEV)
    moe.moe_balance_loss_bwd(dev(z), f, k, 0.5, 0.25, seq_offsets=dev(off),
                             token_mask=dev(live.astype(np.uint8)), out=d)
    compare(f, d, ref, E)
    assert (d.cpu().numpy()[junk] == 0).all()


@gpu
def test_masked_experts_and_rows_without_any():
    """Experts at -inf or at the lowest fp32 value, rows of -inf alone, large logits; choices of
    -1 are skipped."""
    rng = np.random.default_rng(6)
    T, E, k = 64, 20, 3
    z = (rng.standard_normal((T, E)) * 30).astype(np.float32)
    idx = np.argsort(-z, axis=1)[:, :k].astype(np.int32)
    z[:, 5] = -np.inf
    z[:, 6] = np.finfo(np.float32).min
    z[10:13] = -np.inf
    idx[10:13] = -1
    ref = reference(z, idx, k, np.array([0, T]), np.ones(T, bool), 0.5, 0.25)
    f = moe.moe_balance_loss(dev(z), dev(idx), 0.5, 0.25)
    d = moe.moe_balance_loss_bwd(dev(z), f, k, 0.5, 0.25)
    compare(f, d, ref, E)


@gpu
def test_nothing_live():
    z, idx = torch.randn(50, 8, device=DEV), torch.zeros(50, 2, dtype=torch.int32, device=DEV)
    f = moe.moe_balance_loss(z, idx, 1.0, 1.0, token_mask=torch.zeros(50, dtype=torch.uint8, device=DEV))
    d = moe.moe_balance_loss_bwd(z, f, 2, 1.0, 1.0, token_mask=torch.zeros(50, dtype=torch.uint8, device=DEV))
    assert not f["loss"].any() and not f["counts"].any() and not f["tokens"].any() and not d.any()
    e = moe.moe_balance_loss(z[:0], idx[:0], 1.0, 1.0)
    assert not e["loss"].any() and not e["counts"].any() and not e["tokens"].any()
    assert not e["prob_sum"].any()


@gpu
@pytest.mark.parametrize("E,T", [(8, 511), (32, 512), (32, 513), (33, 256), (64, 257), (65, 31), (128, 129),
                                 (132, 64), (256, 65), (256, 3)])
@pytest.mark.parametrize("gaps", [False, True])
def test_few_tokens(E, T, gaps):
    """Both sides of where one workgroup does the whole loss; sequences that are empty, first, last
    and in the middle, and rows before the first and behind the last."""
    rng = np.random.default_rng(E * T)
    z = rng.standard_normal((T, E)).astype(np.float32) * 3
    k = min(E, 5)
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    idx[T // 2] = -1
    live = rng.random(T) >= 0.2
    cut = max(1, T // 3)
    off = np.array([1, 1, cut, T - 1, T - 1] if gaps else [0, T], np.int32)
    ref = reference(z, idx, k, off, live, 0.02, 0.003)
    f = moe.moe_balance_loss(dev(z), dev(idx), 0.02, 0.003, seq_offsets=dev(off),
                             token_mask=dev(live.astype(np.uint8)))
    d = moe.moe_balance_loss_bwd(dev(z), f, k, 0.02, 0.003, seq_offsets=dev(off),
                                 token_mask=dev(live.astype(np.uint8)))
    compare(f, d, ref, E)


@gpu
@pytest.mark.parametrize("S", [1, 3, 40])
def test_no_tokens(S):
    z, idx = torch.zeros(0, 12, device=DEV), torch.zeros(0, 2, dtype=torch.int32, device=DEV)
    off = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    out = {n: torch.full(shape, 7, dtype=dt, device=DEV) for n, shape, dt in (
        ("counts", (S, 12), torch.int32), ("prob_sum", (S, 12), torch.float32),
        ("tokens", (S + 1,), torch.int32), ("loss", (3,), torch.float32))}
    f = moe.moe_balance_loss(z, idx, 1.0, 1.0, seq_offsets=off, out=out)
    assert not any(f[n].any() for n in out)


@gpu
def test_no_gradient_without_imbalance():
    """Even counts: the balance gradient is p (c - c) = 0 up to rounding of sum p."""
    E = 16
    z = torch.randn(E, E, device=DEV)
    idx = torch.arange(E, dtype=torch.int32, device=DEV).reshape(E, 1)
    f = moe.moe_balance_loss(z, idx, 1.0)
    d = moe.moe_balance_loss_bwd(z, f, 1, 1.0)
    # kb c |1 - sum p| <= (1/E) (E + 128) u
    assert d.abs().max() <= (E + 136) * U24 / E


@gpu
def test_more_than_2_to_31_bytes_of_logits():
    T, E, k = (1 << 21) + 77, 256, 1
    g = torch.Generator(device=DEV).manual_seed(3)
    z = torch.randn((T, E), generator=g, device=DEV)
    idx = z.argmax(dim=1, keepdim=True).to(torch.int32)
    f = moe.moe_balance_loss(z, idx, 1.0, 1.0)
    d = moe.moe_balance_loss_bwd(z, f, k, 1.0, 1.0)
    assert torch.equal(f["counts"][0].long(), torch.bincount(idx[:, 0].long(), minlength=E))
    q = torch.zeros(E, dtype=torch.float64, device=DEV)
    for a in range(0, T, 1 << 18):
        q += torch.softmax(z[a:a + (1 << 18)].double(), dim=1).sum(dim=0)
    # 512 chunks of C rows, each summed by 32 lanes groups in turn: C + 512 terms follow one another
    assert ((f["prob_sum"][0].double() - q).abs() <= (T // 512 + 600 + 400) * U24 * q).all()
    p = torch.softmax(z[-4:].double(), dim=1)
    c, lse = f["counts"][0].double(), torch.logsumexp(z[-4:].double(), dim=1)
    ref = p * (E / T / T * (c - (p @ c)[:, None]) + 2 / T * lse[:, None])
    mag = p * (E / T / T * (c + (p @ c)[:, None]) + 2 / T * lse.abs()[:, None])
    assert ((d[-4:].double() - ref).abs() <= 4 * (128 + E + 16) * U24 * mag).all()


@gpu
@pytest.mark.parametrize("T,S", [(3000, 5), (150, 2), (400, 90)])
def test_captured_and_on_another_stream(T, S):
    rng = np.random.default_rng(9)
    E, k = 64, 4
    off = dev(offsets_of(rng, T, S))
    z = torch.randn(T, E, device=DEV)
    idx = z.topk(k, dim=1).indices.to(torch.int32)
    f = moe.moe_balance_loss(z, idx, 0.1, 0.1, seq_offsets=off)
    d = moe.moe_balance_loss_bwd(z, f, k, 0.1, 0.1, seq_offsets=off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_balance_loss(z, idx, 0.1, 0.1, seq_offsets=off, ws=f["ws"], out=f)
        moe.moe_balance_loss_bwd(z, f, k, 0.1, 0.1, seq_offsets=off, out=d)
    side = torch.cuda.Stream()
    for _ in range(4):
        z.normal_()
        idx.copy_(z.topk(k, dim=1).indices)
        f["loss"].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            e = moe.moe_balance_loss(z, idx, 0.1, 0.1, seq_offsets=off)
            h = moe.moe_balance_loss_bwd(z, e, k, 0.1, 0.1, seq_offsets=off)
        side.synchronize()
        for n in ("loss", "counts", "prob_sum", "lse", "tokens"):
            assert torch.equal(e[n], f[n]), n
        assert torch.equal(h, d)


@gpu
def test_binding_refusals():
    z, idx = torch.zeros(6, 8, device=DEV), torch.zeros(6, 2, dtype=torch.int32, device=DEV)
    for bad in (dict(logits=z.bfloat16()), dict(topk_idx=idx.long()), dict(topk_idx=idx[:5]),
                dict(logits=torch.zeros(8, 6, device=DEV).t()), dict(token_mask=torch.ones(6, device=DEV)),
                dict(token_mask=torch.ones(5, dtype=torch.uint8, device=DEV)),
                dict(seq_offsets=torch.tensor([0, 6], dtype=torch.int32)),
                dict(seq_offsets=torch.tensor([0, 6], device=DEV)),
                dict(out={"loss": torch.zeros(2, device=DEV)}),
                dict(ws=torch.zeros(16, dtype=torch.uint8, device=DEV))):
        a = dict(logits=z, topk_idx=idx, balance_coef=0.1)
        with pytest.raises(ValueError):
            moe.moe_balance_loss(**{**a, **bad})


@gpu
@pytest.mark.parametrize("dtype,T,H,E,k", [("f32", 37, 64, 6, 2), ("bf16", 130, 128, 64, 4),
                                           ("bf16", 257, 192, 20, 3), ("bf16", 65, 64, 256, 8),
                                           ("f32", 1, 4, 130, 32), ("bf16", 1, 64, 8, 1)])
def test_route_bwd_add(dtype, T, H, E, k):
    """d_logits within the rounding of one subtraction chain, dx and dw within 2^-14 of the sum of
    absolute terms (the two bf16 halves; moe_route_bwd's bound)."""
    rng = np.random.default_rng(T + E)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, w = dev(rng.standard_normal((T, H)), dt), dev(rng.standard_normal((H, E)) / 8, dt)
    z = rng.standard_normal((T, E))
    idx = np.argsort(-z, axis=1)[:, :k].astype(np.int32)
    gate = rng.random((T, k)).astype(np.float32)
    gate /= gate.sum(axis=1, keepdims=True)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    add = (rng.standard_normal((T, E)) * 0.1).astype(np.float32)
    o = moe.moe_route_bwd_add(dev(dw), dev(gate), dev(idx), dev(add), x, w)
    inner = (gate.astype(np.float64) * dw).sum(axis=1, keepdims=True)
    dz = add.astype(np.float64)
    np.add.at(dz, (np.arange(T)[:, None], idx), gate * (dw - inner))
    mag = np.abs(add) + 0.0
    np.add.at(mag, (np.arange(T)[:, None], idx), gate * (np.abs(dw) + (gate * np.abs(dw)).sum(axis=1, keepdims=True)))
    got = o["d_logits"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - dz) <= (k + 8) * U24 * mag).all()
    xh, wh = x.double().cpu().numpy(), w.double().cpu().numpy()
    for name, ref, m in (("dx_router", dz @ wh.T, mag @ np.abs(wh).T), ("dw_router", xh.T @ dz, np.abs(xh).T @ mag)):
        assert (np.abs(o[name].cpu().numpy() - ref) <= 2.0 ** -14 * m + 1e-30).all(), name
    # in place of the addition, and the same call without it equals moe_route_bwd's logit gradient
    a2 = dev(add)
    o2 = moe.moe_route_bwd_add(dev(dw), dev(gate), dev(idx), a2, x, w, out={"d_logits": a2})
    assert torch.equal(o2["d_logits"], o["d_logits"]) and torch.equal(o2["dw_router"], o["dw_router"])
    zero = moe.moe_route_bwd_add(dev(dw), dev(gate), dev(idx), torch.zeros_like(a2), x, w)
    if not (dtype == "bf16" and E % 4):
        assert torch.equal(zero["d_logits"], moe.moe_route_bwd(dev(dw), dev(gate), dev(idx), x, w)["d_logits"])


@gpu
def test_binding_refusals_of_whole_calls():
    """Calls that give every tensor: as they are they pass, with any one tensor of another type, shape,
    device or order they are refused."""
    z = torch.randn(6, 8, device=DEV)
    a = dict(logits=z, topk_idx=z.topk(2, dim=1).indices.int(), balance_coef=0.1, z_coef=0.2,
             seq_offsets=torch.tensor([0, 2, 6], dtype=torch.int32, device=DEV),
             token_mask=torch.ones(6, dtype=torch.uint8, device=DEV))
    want = moe.moe_balance_loss(**a)
    out = {n: torch.empty_like(t) for n, t in want.items() if n != "ws"}
    a.update(ws=want["ws"], out=out)
    got = moe.moe_balance_loss(**a)
    assert got["ws"] is a["ws"] and all(got[n] is out[n] and torch.equal(got[n], want[n]) for n in out)
    b = {n: a[n] for n in ("logits", "balance_coef", "z_coef", "seq_offsets", "token_mask")}
    b.update(fwd=got, k=2, d_loss=torch.ones(1, device=DEV), out=torch.empty(6, 8, device=DEV))
    d = moe.moe_balance_loss_bwd(**{**b, "out": None})
    assert moe.moe_balance_loss_bwd(**b) is b["out"] and torch.equal(b["out"], d)

    def bad(t):
        yield t.cpu()
        yield t.double()
        yield t[1:]
        if t.numel() > 1:  # (one element is dense at any stride)
            yield torch.stack([t, t], -1)[..., 0]
        yield t.unsqueeze(0)

    def refused(call, args):
        with pytest.raises(ValueError):
            call(**args)

    for call, args, inner in ((moe.moe_balance_loss, a, "out"), (moe.moe_balance_loss_bwd, b, "fwd")):
        for name, t in args.items():
            if torch.is_tensor(t) and name != "ws":
                for u in bad(t):
                    refused(call, {**args, name: u})
        for name in ("lse", "counts", "tokens") + (("loss", "prob_sum") if inner == "out" else ()):
            for u in bad(args[inner][name]):
                refused(call, {**args, inner: {**args[inner], name: u}})
    for u in (a["ws"].cpu(), a["ws"][:16], torch.stack([a["ws"]] * 2, -1)[:, 0]):
        refused(moe.moe_balance_loss, {**a, "ws": u})


@gpu
@pytest.mark.parametrize("E", [3, 32, 60, 128, 132, 256])
@pytest.mark.parametrize("shift", [4096.0, -4096.0])
def test_gradient_of_shifted_logits(E, shift):
    """A softmax does not depend on a shift of its row.  Logits that are multiples of 2^-10 below 2^4
    are shifted by 2^12 without rounding, so without a z loss the gradient has the same bits.  Its own
    bound: z - top is exact here, exp within 4 u, sums of E terms in a tree of at most 13 levels, p and
    sum p c then within 24 and 40 u, the factors 16 more: 80 u of the magnitudes."""
    rng = np.random.default_rng(E)
    T, k = 300, min(E, 4)
    z = np.clip(np.round(rng.standard_normal((T, E)) * 2048) / 1024, -15, 15).astype(np.float32)
    idx = np.argsort(-z, axis=1, kind="stable")[:, :k].astype(np.int32)
    off = np.array([0, 100, 280, 300], np.int32)
    cb = np.float32(0.125)
    d = []
    for a in (z, z + np.float32(shift)):
        f = moe.moe_balance_loss(dev(a), dev(idx), 0.125, seq_offsets=dev(off))
        d.append(moe.moe_balance_loss_bwd(dev(a), f, k, 0.125, seq_offsets=dev(off)))
    ref = reference(z, idx, k, off, np.ones(T, bool), cb, 0.0)
    for got in d:
        err = np.abs(got.cpu().numpy() - ref["d_logits"])
        assert (err <= 80 * U24 * ref["mag"] + 2.0 ** -126).all(), (err / np.maximum(ref["mag"], 1e-30)).max() / U24
    assert torch.equal(d[0], d[1])


def test_sizes_past_one_launch_are_refused():
    """A launch has fewer than 2^32 threads.  The gradient: 256 for a batch of 128 tokens (up to 32
    experts), 64, 32 or 16 (above 128).  The sums: 1024 for 64 experts of a sequence.  The router
    backward: 64 for a token."""
    big = 1 << 50
    for E, T in ((33, (1 << 30) - 64), (65, (1 << 29) - 32), (129, (1 << 28) - 16), (256, (1 << 28) - 16)):
        assert L.moe_balance_loss_bwd(A, A, A, A, N, N, N, T + 1, E, 1, 1, 0.1, 0.1, 0, A, STREAM) == -2, E
        assert "2^32" in _err()
    for E in (193, 256):
        assert L.moe_balance_loss(A, A, A, N, 64, E, 1, 1 << 20, 0.1, 0.1, A, A, A, A, A, A, big, STREAM) == -2
        assert "2^32" in _err()
        assert L.moe_balance_ws_bytes(64, E, 1 << 20) == -2 and L.moe_balance_ws_bytes(64, E, (1 << 20) - 1) > 0
    assert L.moe_balance_ws_bytes(64, 192, 1 << 20) > 0 and L.moe_balance_ws_bytes(64, 8, 1 << 20) > 0
    assert L.moe_route_bwd_add(A, A, A, A, A, A, (1 << 26) - 3, 4, 1, 1, F32, A, N, N, A, big, STREAM) == -2
    assert "2^32" in _err()


@gpu
@pytest.mark.parametrize("T,E,S,drop", [(5000, 128, 1, 0.0), (20000, 256, 40, 0.1), (262144, 64, 3, 0.2),
                                        (400, 32, 2, 0.3), (6000, 16, 900, 0.0), (33, 1, 1, 0.0)])
def test_no_row_is_lost(T, E, S, drop):
    """Rows of equal logits, E a power of two: every probability is 1 / E, and the sums n_s / E are exact
    in any order."""
    rng = np.random.default_rng(T)
    z = np.repeat(rng.standard_normal((T, 1)).astype(np.float32), E, axis=1)
    idx = rng.integers(0, E, (T, 1)).astype(np.int32)
    off = offsets_of(rng, T, S) if S > 1 else np.array([0, T], np.int32)
    live = rng.random(T) >= drop
    f = moe.moe_balance_loss(dev(z), dev(idx), 1.0, seq_offsets=dev(off), token_mask=dev(live.astype(np.uint8)))
    n = np.array([live[off[s]:off[s + 1]].sum() for s in range(S)])
    assert np.array_equal(f["tokens"].cpu().numpy(), np.append(n, n.sum()))
    assert np.array_equal(f["prob_sum"].cpu().numpy(), np.repeat(n[:, None] / E, E, axis=1).astype(np.float32))
    want = np.stack([np.bincount(idx[off[s]:off[s + 1], 0][live[off[s]:off[s + 1]]], minlength=E) for s in range(S)])
    assert np.array_equal(f["counts"].cpu().numpy(), want)


def test_workspace_of_the_most_tokens():
    """1024 chunks and the sequences at most, up to the largest T."""
    for T in (0x7FFF0000, 0x7FFF0000 - 65536, (1 << 31) - (1 << 21), 1 << 28):
        for E in (1, 8, 33, 65, 200):
            assert 0 < L.moe_balance_ws_bytes(T, E, 3) <= 8 * (1030 * (E + 4) + 64 * E), (T, E)


@gpu
def test_the_most_tokens():
    """T k = 0x7fff0000: the last chunk ends near 2^31.  Equal logits of two experts: p = 1/2, sums of
    halves exact up to 2^24 a thread and then as multiples of a chunk's."""
    T = 0x7FFF0000
    z = torch.zeros((T, 2), device=DEV)
    idx = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    idx[-3:] = 1
    f = moe.moe_balance_loss(z, idx, 1.0)
    assert f["counts"].tolist() == [[T - 3, 3]] and f["tokens"].tolist() == [T, T]
    assert f["prob_sum"].tolist() == [[T / 2, T / 2]]
    assert abs(float(f["loss"][0]) - 1.0) < 1e-6
    del f["lse"]
    f["lse"] = torch.full((T,), 0.6931472, device=DEV)
    d = moe.moe_balance_loss_bwd(z, f, 1, 1.0)
    # p (E / (k N n) (c - sum p c)) = 1/2 2 / T^2 (+-)(c0 - c1) / 2
    want = (T - 6) / 2 / T / T
    for rows in (d[:2], d[T // 2:T // 2 + 2], d[-2:]):
        assert ((rows.double() - torch.tensor([want, -want], device=DEV)).abs() <= 8 * U24 * want).all()
