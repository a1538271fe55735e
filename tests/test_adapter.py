"""Low-rank adapters (moe_adapter_fwd, moe_adapter_bwd, moe_adapter_rows) against float64
definitions.

Tolerances (u = 2^-24; e = eps / 2 of the type: half a rounding step relative to the value):
  v   fp32 sum of K products (products of bf16 values are exact) and the scale: (K + 8) u sum |.|
  y   v's error through B; 2^-16 relative for v's own bits (bf16 only; test_rank_values_keep_all_bits
      asks for all of them); the sum of rank products: (2 rank + 8) u; then one rounding: e |y| + u |y|
  dx  the same with N products in w
  dA  w's error through x; the sum of n rows of (three times, for the parts) products:
      (3 n + 16) u; dB the same with v
Values below the normal range of the parts may be lost: 1e-30 absolute."""
import ctypes

import numpy as np
import pytest
import torch

from test_abi_cpu import A, BF16, EINVAL, EUNSUP, EWS, F32, L, N, OK, S as STREAM, U, _err
import moe_expert_layer_router_amd as moe

DEV = torch.device("cuda:0")
U24 = 2.0 ** -24
gpu = pytest.mark.gpu


def definition(x, src, ids, Aw, Bw, scale, y, dy=None, dx=None):
    """Results and error bounds in 64 bits, adapter by adapter (torch, on the inputs' device)."""
    n_ids, rank, K = Aw.shape
    N_ = Bw.shape[1]
    halves = 2.0 ** -16 if Aw.dtype == torch.bfloat16 else 0.0
    d = lambda t: None if t is None else t.double()
    x, Aw, Bw, y, dy, dx = d(x), d(Aw), d(Bw), d(y), d(dy), d(dx)
    sc = torch.ones(n_ids, dtype=torch.float64, device=x.device) if scale is None else scale.double()
    R = ids.numel()
    o = dict(y=y.clone(), v=torch.zeros(R, rank, dtype=torch.float64, device=x.device))
    b = {n: torch.zeros_like(t) for n, t in o.items()}
    if dy is not None:
        o.update(dx=dx.clone(), dA=torch.zeros_like(Aw), dB=torch.zeros_like(Bw))
        b.update({n: torch.zeros_like(o[n]) for n in ("dx", "dA", "dB")})
    rows_x = torch.arange(R, device=x.device) if src is None else src.long()
    valid = (rows_x >= 0) & (rows_x < x.shape[0])
    for a in range(n_ids):
        r = torch.nonzero((ids == a) & valid).squeeze(1)
        if r.numel() == 0:
            continue
        xr, s = x[rows_x[r]], sc[a]
        v = s * (xr @ Aw[a].t())
        ev = (K + 8) * U24 * s.abs() * (xr.abs() @ Aw[a].abs().t())
        o["v"][r], b["v"][r] = v, ev
        o["y"][r] += v @ Bw[a].t()
        b["y"][r] = ev @ Bw[a].abs().t() + (halves + (2 * rank + 8) * U24) * (v.abs() @ Bw[a].abs().t())
        if dy is None:
            continue
        g = dy[r]
        w = s * (g @ Bw[a])
        ew = (N_ + 8) * U24 * s.abs() * (g.abs() @ Bw[a].abs())
        o["dx"][r] += w @ Aw[a]
        b["dx"][r] = ew @ Aw[a].abs() + (halves + (2 * rank + 8) * U24) * (w.abs() @ Aw[a].abs())
        n = 3 * r.numel() + 16
        o["dA"][a] = w.t() @ xr
        b["dA"][a] = (ew + n * U24 * w.abs()).t() @ xr.abs()
        o["dB"][a] = g.t() @ v
        b["dB"][a] = g.abs().t() @ (ev + n * U24 * v.abs())
    return o, b


def within(got, ref, bound, e, name):
    err = (got.double() - ref).abs()
    lim = bound + (e + U24) * ref.abs() * (1 + e) + 1e-30
    bad = err > lim
    assert not bad.any(), f"{name}: {int(bad.sum())} over, worst {float((err / lim).max()):.3g} of the bound"


def make(dtype, R, K, N_, n_ids, rank, order, gather, seed, pitch=0, scaled=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rnd = lambda *s, std=1.0: (torch.randn(s, generator=g, device=DEV) * std).to(dt)
    ids = torch.randint(-1, n_ids, (R,), generator=g, device=DEV, dtype=torch.int32)
    if order == "sorted":
        ids = torch.sort(ids).values
    elif order == "one":
        ids.fill_(n_ids // 2)
    elif order == "none":
        ids.fill_(-1)
    elif order == "range":  # ids outside the adapters
        ids[::3] = n_ids
        ids[1::5] = -2 ** 31
        ids[2::7] = 2 ** 31 - 1
    ids = ids.contiguous()
    x_rows = max(1, R // 3) if gather else R
    src = None
    if gather:
        src = torch.randint(0, x_rows, (R,), generator=g, device=DEV, dtype=torch.int32)
        if R > 4:
            src[1], src[-1], src[R // 2] = -1, x_rows, 2 ** 31 - 1
    wide = lambda rows, cols: rnd(rows, cols + pitch)[:, :cols]
    return dict(x=wide(x_rows, K), src=src, ids=ids, A=rnd(n_ids, rank, K, std=K ** -0.5),
                B=rnd(n_ids, N_, rank, std=rank ** -0.5),
                scale=torch.rand(n_ids, generator=g, device=DEV) + 0.5 if scaled else None,
                y=wide(R, N_), dy=wide(R, N_), dx=wide(R, K),
                e=torch.finfo(dt).eps / 2 if dtype == "bf16" else U24)


def check(s, accumulate=False, backward=True):
    base = {n: s[n].clone() for n in ("y", "dx")}
    ids_before = s["ids"].clone()
    args = (s["x"], s["src"], s["ids"], s["A"], s["B"], s["scale"], base["y"], s["dy"], base["dx"])
    o, b = definition(*args)
    v = moe.moe_adapter_fwd(s["x"], s["ids"], s["A"], s["B"], s["y"], scale=s["scale"], src_row=s["src"],
                            want_v=True)
    untouched = o["v"].abs().sum(dim=1) == 0
    within(v, o["v"], b["v"], 0.0, "v")
    within(s["y"], o["y"], b["y"], s["e"], "y")
    assert torch.equal(s["y"][untouched], base["y"][untouched]) and not v[untouched].any()
    if not backward:
        return
    out = None
    if accumulate:
        out = {"dA": torch.full_like(s["A"], 0.5, dtype=torch.float32),
               "dB": torch.full_like(s["B"], -0.5, dtype=torch.float32)}
    r = moe.moe_adapter_bwd(s["dy"], s["x"], s["ids"], s["A"], s["B"], v, s["dx"], scale=s["scale"],
                            src_row=s["src"], accumulate=accumulate, out=out)
    within(s["dx"], o["dx"], b["dx"], s["e"], "dx")
    assert torch.equal(s["dx"][untouched], base["dx"][untouched])
    for n, add in (("dA", 0.5), ("dB", -0.5)):
        ref = o[n] + add if accumulate else o[n]
        within(r[n], ref, b[n] + (8 * U24 if accumulate else 0.0), 0.0, n)
    if not accumulate:
        unused = [a for a in range(s["A"].shape[0]) if not (s["ids"] == a).any()]
        assert not r["dA"][unused].any() and not r["dB"][unused].any()
        r2 = moe.moe_adapter_bwd(s["dy"], s["x"], s["ids"], s["A"], s["B"], v, None, scale=s["scale"],
                                 src_row=s["src"])
        assert torch.equal(r["dA"], r2["dA"]) and torch.equal(r["dB"], r2["dB"])  # the same bits
    assert torch.equal(s["ids"], ids_before)


# ---------------------------------------------------------------------------
# no GPU
# ---------------------------------------------------------------------------

def test_refusals():
    big = 1 << 40
    f = L.moe_adapter_fwd
    ok = [A, N, A, A, A, N, 16, 16, 64, 64, 64, 64, 4, 16, BF16, A, N, STREAM]

    def fwd(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert fwd(_6=-1) == EINVAL and fwd(_7=-1) == EINVAL
    assert fwd(_6=2 ** 31 - 1, _7=2 ** 31 - 1) == EUNSUP
    assert fwd(_8=0) == EINVAL and fwd(_8=60) == EINVAL and fwd(_9=63) == EINVAL
    assert fwd(_10=56) == EINVAL and "ldx" in _err()
    assert fwd(_10=65) == EINVAL and fwd(_11=60) == EINVAL and "ldy" in _err()
    assert fwd(_12=0) == EINVAL and fwd(_13=0) == EINVAL and fwd(_14=5) == EINVAL
    assert fwd(_13=12) == EUNSUP and fwd(_13=136) == EUNSUP and "rank" in _err()
    assert fwd(_8=1 << 21, _10=1 << 21) == EUNSUP and fwd(_12=(1 << 20) + 1) == EUNSUP
    for i, name in ((0, "x"), (2, "row_id"), (3, "A"), (4, "B"), (15, "y")):
        assert fwd(**{f"_{i}": N}) == EINVAL and name in _err()
    for i in (0, 3, 4, 15, 16):
        assert fwd(**{f"_{i}": U}) == EINVAL and "aligned" in _err()
    assert fwd(_6=0, _0=N, _2=N, _15=N) == OK
    g = L.moe_adapter_bwd
    okb = [A, A, N, A, A, A, A, N, 16, 16, 64, 64, 64, 64, 64, 4, 16, BF16, A, A, A, 0, A, big, STREAM]

    def bwd(**kw):
        a = list(okb)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return g(*a)

    assert bwd(_15=257) == EUNSUP and "256" in _err()
    assert bwd(_21=2) == EINVAL and "accumulate" in _err()
    assert bwd(_19=N) == EINVAL and "together" in _err()
    assert bwd(_14=56) == EINVAL and "lddx" in _err()
    assert bwd(_6=N) == EINVAL and "v must" in _err()
    for i, name in ((0, "dy"), (1, "x"), (3, "row_id"), (4, "A"), (5, "B")):
        assert bwd(**{f"_{i}": N}) == EINVAL and name in _err()
    assert bwd(_22=N) == EWS and bwd(_23=64) == EWS and bwd(_22=U) == EINVAL
    assert bwd(_16=20) == EUNSUP and bwd(_12=62) == EINVAL
    w = L.moe_adapter_ws_bytes
    assert w(-1, 64, 64, 4, 16, BF16) == EINVAL and w(16, 64, 64, 257, 16, BF16) == EUNSUP
    assert w(0, 64, 64, 4, 16, F32) > 0 and w(16, 64, 64, 4, 16, 2) == EINVAL
    r = L.moe_adapter_rows
    assert r(A, A, A, 0, 8, 2, 16, A, STREAM) == EINVAL and r(A, A, A, 257, 8, 2, 16, A, STREAM) == EINVAL
    assert r(A, A, A, 4, -1, 2, 16, A, STREAM) == EINVAL and r(A, A, A, 4, 8, 2, -1, A, STREAM) == EINVAL
    assert r(A, A, A, 256, 8, 1 << 23, 16, A, STREAM) == EINVAL and r(A, A, A, 4, 8, -1, 16, A, STREAM) == EINVAL
    for i, name in ((0, "offsets"), (1, "src_row"), (2, "token_adapter"), (7, "row_id")):
        a = [A, A, A, 4, 8, 2, 16, A, STREAM]
        a[i] = N
        assert r(*a) == EINVAL and name in _err()
    assert r(N, N, N, 4, 8, 2, 0, N, STREAM) == OK


def test_shared_memory_is_refused():
    """x and y (dy and dx, x and dx) that share an element; columns of one wider matrix do not."""
    at = lambda n: A.value + n
    fwd = lambda x, ldx, y, ldy, K=64, N_=64, R=16: L.moe_adapter_fwd(
        x, N, A, A, A, N, R, R, K, N_, ldx, ldy, 4, 16, BF16, y, N, STREAM)
    assert fwd(A, 64, A, 64) == EINVAL and "overlap" in _err()
    assert fwd(A, 64, at(16 * 64 * 2 - 16), 64) == EINVAL and "overlap" in _err()
    assert fwd(A, 128, at(112), 128) == EINVAL and "overlap" in _err()       # columns 0..63 and 56..119
    assert fwd(A, 128, at(144), 128) == EINVAL and "overlap" in _err()       # y's last columns in the next row
    assert fwd(A, 128, at(256 * 3 + 16), 128) == EINVAL and "overlap" in _err()
    assert fwd(A, 72, at(128), 136) == EINVAL and "overlap" in _err()        # two pitches
    big = 1 << 40
    bwd = lambda dy, x, dx: L.moe_adapter_bwd(dy, x, N, A, A, A, A, N, 16, 16, 64, 64, 64, 64, 64, 4, 16,
                                              BF16, dx, A, A, 0, A, big, STREAM)
    far = at(1 << 20)
    assert bwd(A, far, A) == EINVAL and "dy and dx" in _err()
    assert bwd(far, A, at(32)) == EINVAL and "x and dx" in _err()


def test_definition_gradient_matches_differences():
    """dA, dB, dx of the definition against central differences of <dy, y> in 64 bits."""
    g = torch.Generator().manual_seed(1)
    R, K, N_, n_ids, rank = 7, 5, 6, 3, 2
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    x, Aw, Bw, dy = rnd(R, K), rnd(n_ids, rank, K), rnd(n_ids, N_, rank), rnd(R, N_)
    sc, ids = rnd(n_ids), torch.tensor([0, 2, -1, 2, 0, 2, 2])
    zero_y, zero_x = torch.zeros(R, N_), torch.zeros(R, K)
    f = lambda x, Aw, Bw: float((definition(x, None, ids, Aw, Bw, sc, zero_y)[0]["y"] * dy).sum())
    o, _ = definition(x, None, ids, Aw, Bw, sc, zero_y, dy, zero_x)
    for name, t, at in (("dx", x, 0), ("dA", Aw, 1), ("dB", Bw, 2)):
        for i in range(t.numel()):
            h = torch.zeros_like(t).view(-1)
            h[i] = 1e-5
            a, c = [x, Aw, Bw], [x, Aw, Bw]
            a[at], c[at] = t + h.view_as(t), t - h.view_as(t)
            # linear in each of the three: the rounding of f over h alone
            assert abs((f(*a) - f(*c)) / 2e-5 - float(o[name].reshape(-1)[i])) < 1e-8


# ---------------------------------------------------------------------------
# on the GPU
# ---------------------------------------------------------------------------

CASES = [  # dtype, R, K, N, n_ids, rank, order, gather, pitch, scaled
    ("bf16", 1, 8, 8, 1, 8, "one", False, 0, True), ("bf16", 1, 2048, 2048, 40, 16, "one", False, 0, True),
    ("f32", 1, 4, 4, 1, 8, "one", False, 0, False), ("bf16", 3, 40, 24, 2, 16, "mixed", False, 8, True),
    ("bf16", 16, 64, 64, 3, 24, "none", False, 0, True), ("bf16", 100, 72, 200, 300, 16, "mixed", False, 0, True),
    ("f32", 65, 36, 68, 5, 40, "mixed", True, 4, True), ("bf16", 257, 768, 520, 7, 64, "sorted", True, 0, False),
    ("bf16", 511, 136, 1032, 4, 128, "mixed", False, 16, True), ("f32", 700, 260, 516, 9, 64, "sorted", False, 0, True),
    ("bf16", 1025, 256, 256, 250, 8, "mixed", True, 0, True), ("bf16", 5000, 128, 192, 16, 16, "sorted", False, 0, True),
    ("bf16", 20000, 64, 72, 3, 32, "range", False, 0, True), ("bf16", 33000, 64, 64, 2, 16, "one", True, 0, True),
    ("f32", 20001, 64, 40, 6, 8, "sorted", False, 0, True), ("bf16", 17000, 96, 64, 5, 120, "sorted", False, 0, True),
    ("f32", 33333, 32, 36, 256, 16, "mixed", False, 0, True), ("bf16", 40000, 200, 128, 8, 64, "mixed", False, 0, True),
    ("bf16", 3000, 64, 72, 255, 16, "mixed", True, 0, True), ("bf16", 9001, 72, 136, 40, 128, "mixed", False, 0, True),
    ("f32", 1800, 40, 36, 100, 120, "mixed", True, 0, True),
]


@gpu
@pytest.mark.parametrize("dtype,R,K,N_,n_ids,rank,order,gather,pitch,scaled", CASES)
def test_against_definition(dtype, R, K, N_, n_ids, rank, order, gather, pitch, scaled):
    s = make(dtype, R, K, N_, n_ids, rank, order, gather, R + K, pitch, scaled)
    check(s, backward=n_ids <= 256)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,n_ids,rank,order", [(1024, 1, 16, "one"), (1024, 3, 32, "mixed"), (1023, 2, 24, "range"),
                                                (129, 256, 8, "mixed"), (128, 1, 32, "one"), (5, 3, 8, "sorted"),
                                                (1025, 1, 16, "one"), (1024, 2, 40, "mixed")])
def test_gradients_of_few_rows(dtype, R, n_ids, rank, order):
    """Both sides of where an adapter's rows are one sum (1024 rows, rank 32)."""
    for accumulate in (False, True):
        check(make(dtype, R, 72, 136, n_ids, rank, order, R % 2 == 1, R + rank), accumulate=accumulate)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_accumulated_gradients(dtype):
    check(make(dtype, 3001, 64, 136, 4, 16, "sorted", False, 7), accumulate=True)
    check(make(dtype, 90, 64, 136, 4, 16, "mixed", True, 8), accumulate=True)


@gpu
def test_one_request_never_reaches_another():
    """NaN and infinities in one adapter's weights and rows, and around the matrices."""
    s = make("bf16", 200, 128, 136, 4, 16, "mixed", False, 3, pitch=8)
    bad = s["ids"] == 2
    y0 = s["y"].clone()
    v = moe.moe_adapter_fwd(s["x"], s["ids"], s["A"], s["B"], s["y"], scale=s["scale"], want_v=True)
    clean_y, clean_v = s["y"].clone(), v
    clean = moe.moe_adapter_bwd(s["dy"], s["x"], s["ids"], s["A"], s["B"], v, None, scale=s["scale"])
    s["y"].copy_(y0)
    s["A"][2], s["B"][2, ::2], s["B"][2, 1::2] = float("nan"), float("inf"), float("nan")
    s["x"][bad], s["dy"][bad] = float("inf"), float("nan")
    s["x"][s["ids"] == -1] = float("nan")
    v = moe.moe_adapter_fwd(s["x"], s["ids"], s["A"], s["B"], s["y"], scale=s["scale"], want_v=True)
    assert torch.equal(s["y"][~bad], clean_y[~bad]) and torch.equal(v[~bad], clean_v[~bad])
    got = moe.moe_adapter_bwd(s["dy"], s["x"], s["ids"], s["A"], s["B"], v, None, scale=s["scale"])
    for n in ("dA", "dB"):
        for a in (0, 1, 3):
            assert torch.equal(got[n][a], clean[n][a])


@gpu
@pytest.mark.parametrize("dtype,rank", [("bf16", 16), ("f32", 16), ("bf16", 72)])
def test_row_order_changes_no_bit(dtype, rank):
    """Rows sorted by adapter, and the same rows mixed (which are regrouped)."""
    s = make(dtype, 4000, 136, 200, 37, rank, "sorted", False, 12)
    perm = torch.randperm(4000, device=DEV)
    y = s["y"][perm].contiguous()
    v = moe.moe_adapter_fwd(s["x"], s["ids"], s["A"], s["B"], s["y"], scale=s["scale"], want_v=True)
    w = moe.moe_adapter_fwd(s["x"][perm].contiguous(), s["ids"][perm].contiguous(), s["A"], s["B"], y,
                            scale=s["scale"], want_v=True)
    assert torch.equal(s["y"][perm], y) and torch.equal(v[perm], w)


@gpu
def test_columns_past_the_width_are_left_alone():
    s = make("bf16", 130, 64, 72, 3, 16, "mixed", False, 4)
    wide = torch.full((130, 96), 7.0, dtype=torch.bfloat16, device=DEV)
    wide[:, 8:80] = s["y"]
    moe.moe_adapter_fwd(s["x"], s["ids"], s["A"], s["B"], wide[:, 8:80], scale=s["scale"])
    moe.moe_adapter_fwd(s["x"], s["ids"], s["A"], s["B"], s["y"], scale=s["scale"])
    assert torch.equal(wide[:, 8:80], s["y"]) and (wide[:, :8] == 7).all() and (wide[:, 80:] == 7).all()


@gpu
def test_offsets_past_32_bits():
    """Weights, rows and results whose last elements lie past 2^32 bytes."""
    bf = torch.bfloat16
    n_ids, rank, K, N_ = (1 << 15) + 3, 16, 64, 4096
    s = make("bf16", 8, K, N_, 2, rank, "one", False, 5)
    Bw = torch.zeros((n_ids, N_, rank), dtype=bf, device=DEV)
    Aw = torch.zeros((n_ids, rank, K), dtype=bf, device=DEV)
    Aw[-1], Bw[-1] = s["A"][1], s["B"][1]
    ids = torch.full((8,), n_ids - 1, dtype=torch.int32, device=DEV)
    ref = s["y"].clone()
    moe.moe_adapter_fwd(s["x"], s["ids"], s["A"], s["B"], ref)
    moe.moe_adapter_fwd(s["x"], ids, Aw, Bw, s["y"])
    assert torch.equal(ref, s["y"])
    del Aw, Bw
    R = (1 << 20) + 5
    big = make("bf16", 64, 2048, 2056, 2, 8, "one", False, 6)
    y = torch.zeros((R, 2056), dtype=bf, device=DEV)
    x = torch.zeros((R, 2048), dtype=bf, device=DEV)
    x[-64:] = big["x"]
    ids = torch.full((R,), -1, dtype=torch.int32, device=DEV)
    ids[-64:] = 1
    moe.moe_adapter_fwd(x, ids, big["A"], big["B"], y)
    want = torch.zeros((64, 2056), dtype=bf, device=DEV)
    moe.moe_adapter_fwd(big["x"], torch.ones(64, dtype=torch.int32, device=DEV), big["A"], big["B"], want)
    o, b = definition(big["x"], None, torch.ones(64, device=DEV), big["A"], big["B"], None, torch.zeros_like(want))
    within(y[-64:], o["y"], b["y"], 2.0 ** -8, "y")
    assert not y[:-64].any()


@gpu
def test_gradients_not_wanted():
    s = make("bf16", 60, 64, 72, 3, 16, "mixed", False, 9)
    v = moe.moe_adapter_fwd(s["x"], s["ids"], s["A"], s["B"], s["y"], scale=s["scale"], want_v=True)
    dx = s["dx"].clone()
    full = moe.moe_adapter_bwd(s["dy"], s["x"], s["ids"], s["A"], s["B"], v, s["dx"], scale=s["scale"])
    part = moe.moe_adapter_bwd(s["dy"], s["x"], s["ids"], s["A"], s["B"], None, dx, scale=s["scale"], want_dw=False)
    assert torch.equal(dx, s["dx"]) and part["dA"] is None and full["dA"] is not None
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    r = moe.moe_adapter_bwd(s["dy"][:0], s["x"][:0], none, s["A"], s["B"], v[:0], s["dx"][:0])
    assert not r["dA"].any() and not r["dB"].any()


@gpu
@pytest.mark.parametrize("R", [900, 2500, 5000])
def test_captured_and_on_another_stream(R):
    s = make("bf16", R, 128, 136, 12, 16, "mixed", True, 11)
    s["src"].clamp_(0, s["x"].shape[0] - 1)
    y0, dx0 = s["y"].clone(), s["dx"].clone()
    fwd = lambda y, v=None: moe.moe_adapter_fwd(s["x"], s["ids"], s["A"], s["B"], y, scale=s["scale"],
                                                src_row=s["src"], want_v=True, out=v)
    bwd = lambda v, dx, ws=None, out=None: moe.moe_adapter_bwd(
        s["dy"], s["x"], s["ids"], s["A"], s["B"], v, dx, scale=s["scale"], src_row=s["src"], ws=ws, out=out)
    v = fwd(s["y"])
    r = bwd(v, s["dx"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s["y"].copy_(y0)
        s["dx"].copy_(dx0)
        fwd(s["y"], v)
        bwd(v, s["dx"], r["ws"], r)
    side = torch.cuda.Stream()
    for i in range(4):
        s["x"].normal_()
        s["dy"].normal_()
        s["ids"].random_(-1, 12)
        graph.replay()
        torch.cuda.synchronize()
        y, dx = y0.clone(), dx0.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            ve = fwd(y)
            re = bwd(ve, dx)
        side.synchronize()
        assert torch.equal(y, s["y"]) and torch.equal(ve, v) and torch.equal(dx, s["dx"])
        assert torch.equal(re["dA"], r["dA"]) and torch.equal(re["dB"], r["dB"])


@gpu
def test_adapter_rows():
    rng = np.random.default_rng(0)
    T, E, k, lo, hi, n_ad = 301, 16, 4, 4, 13, 5
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    tok = rng.integers(-1, n_ad + 1, T).astype(np.int32)
    x = torch.zeros(T, 8, device=DEV)
    p = moe.moe_permute(x, torch.from_numpy(idx).to(DEV), E, lo, hi, copy_rows=False)
    ids = moe.moe_adapter_rows(p["offsets"], p["src_row"], torch.from_numpy(tok).to(DEV), n_ad).cpu().numpy()
    off = p["offsets"].cpu().numpy()
    src = p["src_row"].cpu().numpy()
    want = np.full(T * k, -1, np.int32)
    for e in range(hi - lo):
        for r in range(off[e], off[e + 1]):
            a = tok[src[r]]
            if 0 <= a < n_ad:
                want[r] = a * (hi - lo) + e
    assert np.array_equal(ids, want) and (want >= 0).any()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_columns_of_one_matrix(dtype):
    """x and y as neighbouring columns of one matrix give the bits of separate ones."""
    s = make(dtype, 37, 64, 72, 3, 16, "mixed", False, 1)
    want = s["y"].clone()
    moe.moe_adapter_fwd(s["x"], s["ids"], s["A"], s["B"], want)
    wide = torch.cat([s["x"], s["y"], s["x"]], 1)
    moe.moe_adapter_fwd(wide[:, :64], s["ids"], s["A"], s["B"], wide[:, 64:136])
    assert torch.equal(wide[:, 64:136], want)
    assert torch.equal(wide[:, :64], s["x"]) and torch.equal(wide[:, 136:], s["x"])
    wide = torch.cat([s["y"], s["x"]], 1)  # y before x
    moe.moe_adapter_fwd(wide[:, 72:], s["ids"], s["A"], s["B"], wide[:, :72])
    assert torch.equal(wide[:, :72], want)


@gpu
def test_no_token_rows():
    """x without rows: every src_row is outside, no row has an adapter."""
    s = make("bf16", 20, 64, 72, 3, 16, "mixed", False, 1)
    none = dict(x=s["x"][:0], src_row=torch.zeros(20, dtype=torch.int32, device=DEV))
    y = s["y"].clone()
    v = moe.moe_adapter_fwd(row_id=s["ids"], A=s["A"], B=s["B"], y=y, want_v=True, **none)
    assert torch.equal(y, s["y"]) and not v.any()
    dx = torch.ones(20, 64, dtype=torch.bfloat16, device=DEV)
    o = moe.moe_adapter_bwd(s["y"], row_id=s["ids"], A=s["A"], B=s["B"], v=v, dx=dx, **none)
    assert (dx == 1).all() and not o["dA"].any() and not o["dB"].any()


@gpu
def test_binding_refusals():
    s = make("bf16", 20, 64, 72, 3, 16, "mixed", False, 1)
    a = dict(x=s["x"], row_id=s["ids"], A=s["A"], B=s["B"], y=s["y"])
    for bad in (dict(x=s["x"].float()), dict(x=s["x"][:19]), dict(row_id=s["ids"].long()), dict(A=s["A"][:2]),
                dict(A=s["A"].float()), dict(y=s["y"][:, :64]), dict(y=s["y"].t().contiguous().t()),
                dict(scale=torch.ones(2, device=DEV)), dict(src_row=torch.zeros(20, device=DEV)),
                dict(row_id=s["ids"].cpu()), dict(x=s["x"].cpu()), dict(A=s["A"].transpose(1, 2)),
                dict(y=torch.zeros(1, 72, dtype=torch.bfloat16, device=DEV).expand(20, 72)),
                dict(want_v=True, out=torch.zeros(20, 8, device=DEV))):
        with pytest.raises(ValueError):
            moe.moe_adapter_fwd(**{**a, **bad})
    with pytest.raises(moe.MoEError, match="ldy"):
        moe.moe_adapter_fwd(**{**a, "y": torch.zeros(20, 73, dtype=torch.bfloat16, device=DEV)[:, :72]})
    with pytest.raises(moe.MoEError, match="rank"):
        moe.moe_adapter_fwd(s["x"], s["ids"], s["A"][:, :12].contiguous(), s["B"][..., :12].contiguous(), s["y"])
    v = moe.moe_adapter_fwd(**a, want_v=True)
    ws = moe.moe_adapter_bwd(s["y"], s["x"], s["ids"], s["A"], s["B"], v, None)["ws"]
    for bad in (ws.cpu(), ws[:64], torch.stack([ws, ws], 1)[:, 0]):
        with pytest.raises(ValueError, match="ws|workspace"):
            moe.moe_adapter_bwd(s["y"], s["x"], s["ids"], s["A"], s["B"], v, None, ws=bad)


def test_ffn_adapter_refusals():
    f = L.moe_grouped_ffn_fwd_adapter
    ok = [A, N, A, A, 4, 16, 16, 64, 64, A, A, A, A, A, N, N, A, A, N, 8, 16, BF16, A, A, A, A, 1 << 30, STREAM]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert call(_6=15) == EINVAL and "x_rows" in _err()
    assert call(_1=A, _21=F32) == EUNSUP and "bf16 only" in _err()
    assert call(_7=96) == EUNSUP and call(_20=20) == EUNSUP and call(_19=0) == EINVAL
    assert call(_13=N) == EINVAL and "together" in _err()
    assert call(_12=U) == EINVAL and "aligned" in _err()
    for i, name in ((0, "x"), (2, "offsets"), (3, "row_id"), (9, "w_gate"), (10, "w_up"), (11, "w_down"),
                    (22, "gu"), (23, "h_perm"), (24, "y_perm")):
        assert call(**{f"_{i}": N}) == EINVAL and name in _err()
    assert call(_25=N) == EWS and call(_26=16) == EWS
    assert call(_5=0, _6=0, _0=N, _3=N, _22=N, _23=N, _24=N) == OK


@gpu
def test_binding_refusals_of_whole_calls():
    """Calls that give every tensor: as they are they pass, with any one tensor of another type, shape,
    device or order they are refused."""
    s = make("bf16", 20, 64, 72, 3, 16, "mixed", True, 1)
    a = dict(x=s["x"], row_id=s["ids"], A=s["A"], B=s["B"], y=s["y"], scale=s["scale"], src_row=s["src"],
             want_v=True, out=torch.zeros(20, 16, device=DEV))
    v = moe.moe_adapter_fwd(**a)
    assert v is a["out"]
    b = {n: a[n] for n in ("x", "row_id", "A", "B", "scale", "src_row")}
    b.update(dy=torch.randn(20, 72, device=DEV).bfloat16(), v=v, dx=torch.zeros(20, 64, device=DEV).bfloat16())
    fresh = moe.moe_adapter_bwd(**{**b, "dx": b["dx"].clone()})
    b.update(ws=fresh["ws"], out={n: torch.zeros_like(fresh[n]) for n in ("dA", "dB")})
    got = moe.moe_adapter_bwd(**b)
    assert all(got[n] is b["out"][n] and torch.equal(got[n], fresh[n]) for n in b["out"])

    def bad(t):
        yield t.cpu()
        yield t.double()
        if t is not a["x"]:  # (with src_row, x may have any number of rows)
            yield t[1:]
        if t is not a["x"] and t is not a["y"] and t is not b["dy"] and t is not b["dx"]:  # (rows at a pitch)
            yield torch.stack([t, t], -1)[..., 0]
        yield t.unsqueeze(0)

    for call, args in ((moe.moe_adapter_fwd, a), (moe.moe_adapter_bwd, b)):
        for name, t in args.items():
            if torch.is_tensor(t) and name != "ws":
                for u in bad(t):
                    with pytest.raises(ValueError):
                        call(**{**args, name: u})
    for name, t in b["out"].items():
        for u in bad(t):
            with pytest.raises(ValueError):
                moe.moe_adapter_bwd(**{**b, "out": {**b["out"], name: u}})
    for u in (b["ws"].cpu(), b["ws"][:64], torch.stack([b["ws"]] * 2, -1)[:, 0]):
        with pytest.raises(ValueError):
            moe.moe_adapter_bwd(**{**b, "ws": u})


def paired(rows, width, n_ids, rank, n_out, g):
    """Whole numbers for x [rows, width], A [n_ids, rank, width], B [n_ids, n_out, rank]: rank values
    2 i and 2 i + 1 are sums of 20 bits or so that differ by one element of x alone, and every
    column of B takes the difference of one such pair.  Every sum is below 2^24 (each product is at
    most 2^14, at most 512 of them), so fp32 holds them all, and a result is an element of x."""
    pick = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV).double()
    x, Aw = pick(-127, 128, rows, width), pick(-127, 128, n_ids, rank, width)
    Aw[:, 1::2] = Aw[:, ::2]
    c = torch.randint(0, width, (n_ids, rank // 2, 1), generator=g, device=DEV)
    Aw[:, 1::2].scatter_add_(2, c, torch.ones_like(c).double())
    Bw = torch.zeros(n_ids, n_out, rank, dtype=torch.float64, device=DEV)
    n = torch.arange(n_out, device=DEV)
    Bw[:, n, 2 * n % rank], Bw[:, n, (2 * n + 1) % rank] = 1.0, -1.0
    return x, Aw, Bw


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 64, 72, 128])
def test_rank_values_keep_all_bits(dtype, rank):
    """Rank values of 20 bits that cancel to 8: exact, forward and data gradients."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device=DEV).manual_seed(rank)
    R, n_ids, wide, out = 77, 3, 512, 136
    ids = torch.randint(-1, n_ids, (R,), generator=g, device=DEV, dtype=torch.int32)
    x, Aw, Bw = paired(R, wide, n_ids, rank, out, g)
    zero = torch.zeros(R, out, dtype=torch.float64, device=DEV)
    want = definition(x, None, ids, Aw, Bw, None, zero)[0]["y"]
    assert want.abs().max() <= 127 and want.any()
    y = zero.to(dt)
    moe.moe_adapter_fwd(x.to(dt), ids, Aw.to(dt), Bw.to(dt), y)
    assert torch.equal(y.double(), want)
    # the data gradients take dy for x, B^T for A and A^T for B
    Ab, Bb = Bw.transpose(1, 2).contiguous(), Aw.transpose(1, 2).contiguous()
    dx = zero.to(dt)
    moe.moe_adapter_bwd(x.to(dt), zero.to(dt), ids, Ab.to(dt), Bb.to(dt), None, dx, want_dw=False)
    assert torch.equal(dx.double(), want)


def test_sizes_past_one_launch_are_refused():
    """A launch has fewer than 2^32 threads.  The adapter kernel: 256 for 16 rows, 32 above rank 64, 128
    for these in fp32 (the tile that fits a CU twice); the FFN's activation: 64 for a row."""
    far = lambda n: A.value + n

    def fwd(R, rank, dtype, K=8):
        return L.moe_adapter_fwd(A, N, A, A, A, N, R, R, K, K, K, K, 4, rank, dtype, far(1 << 46), N, STREAM)

    for rank, dtype, most in ((16, BF16, (1 << 28) - 16), (64, F32, (1 << 28) - 16), (128, BF16, (1 << 29) - 32),
                              (128, F32, (1 << 30) - 32)):
        assert fwd(most + 1, rank, dtype) == EUNSUP and "2^32" in _err(), (rank, dtype)
    big = 1 << 60
    R = (1 << 28) - 16 + 1
    assert L.moe_adapter_bwd(A, A, N, A, A, A, A, N, R, R, 8, 8, 8, 8, 8, 4, 16, BF16, far(1 << 46), A, A, 0, A, big,
                             STREAM) == EUNSUP and "2^32" in _err()
    # the transposed weights: a thread for 4 bytes of columns of 16 bytes of ranks
    w = 1 << 20
    assert L.moe_adapter_bwd(A, A, N, A, A, A, A, N, 4, 4, w, w, w, w, w, 256, 32, F32, far(1 << 46), A, A, 0, A, big,
                             STREAM) == EUNSUP and "2^32" in _err()
    R = (1 << 26) - 3
    assert L.moe_grouped_ffn_fwd_adapter(A, N, A, A, 4, R, R, 4, 4, A, A, A, A, A, N, N, A, A, N, 8, 16, F32, A, A, A,
                                         A, big, STREAM) == EUNSUP and "2^32" in _err()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("row", [0, 3, 19])
def test_one_row_beside_many(dtype, row):
    """x one row of a matrix, behind the columns that y takes of all its rows: they share nothing."""
    s = make(dtype, 20, 64, 72, 3, 16, "mixed", False, 1)
    src = torch.zeros(20, dtype=torch.int32, device=DEV)
    wide = torch.cat([s["y"], s["x"]], 1)
    x = s["x"][row:row + 1].contiguous()
    moe.moe_adapter_fwd(x, s["ids"], s["A"], s["B"], s["y"], src_row=src)
    moe.moe_adapter_fwd(wide[row:row + 1, 72:], s["ids"], s["A"], s["B"], wide[:, :72], src_row=src)
    assert torch.equal(wide[:, :72], s["y"]) and torch.equal(wide[:, 72:], s["x"])
    # one that begins in y's columns, and one that ends in those of the next row
    for first in (8, 64) + ((80,) if row < 19 else ()):
        flat = wide.reshape(-1)[row * 136 + first:row * 136 + first + 64].reshape(1, 64)
        with pytest.raises(moe.MoEError, match="overlap"):
            moe.moe_adapter_fwd(flat, s["ids"], s["A"], s["B"], wide[:, :72], src_row=src)


def test_overlap_of_the_largest_matrices():
    """Extents past 2^63 bytes (as the arguments give them) are compared without overflow."""
    x = ctypes.c_void_p(A.value + (1 << 40))
    for back in (64, 1 << 30, 1 << 38):
        y = ctypes.c_void_p(x.value + back)
        assert L.moe_adapter_fwd(x, A, A, A, A, N, 16, (1 << 31) - 1, 64, 64, (1 << 31) - 8, 64, 4, 16, F32, y, N,
                                 STREAM) == EINVAL and "overlap" in _err()


def whole_numbers(dtype, R, K, N_, n_ids, rank, seed):
    """make() with -1, 0 and 1 for x, y, dx and dy, and four 1 or -1 in each rank value's column of A
    and of B: all results are whole numbers that their types hold."""
    s = make(dtype, R, K, N_, n_ids, rank, "sorted", False, seed, scaled=False)
    g = torch.Generator(device=DEV).manual_seed(seed)
    for n in ("x", "y", "dy", "dx"):
        s[n] = torch.randint(-1, 2, s[n].shape, generator=g, device=DEV).to(s[n].dtype)
    for n, cols in (("A", K), ("B", N_)):
        w = torch.zeros(n_ids, rank, cols, device=DEV)
        at = torch.randint(0, cols, (n_ids, rank, 4), generator=g, device=DEV)
        w.scatter_(2, at, torch.randint(0, 2, at.shape, generator=g, device=DEV).float() * 2 - 1)
        s[n] = (w if n == "A" else w.transpose(1, 2)).contiguous().to(s[n].dtype)
    return s


LONG = [  # R, K, N, n_ids, rank: rows of a chunk of the weight gradients, several chunks an adapter
    (9001, 768, 2048, 16, 16),    # 256
    (9001, 4096, 4096, 5, 8),     # 512
    (20011, 4104, 4096, 9, 32),   # 1024
    (16000, 2048, 1536, 3, 24),   # 384
    (300001, 64, 64, 7, 8),       # 896; a wave orders more than 512 rows
    (40000, 256, 256, 5, 64), (33333, 64, 64, 1, 16), (20001, 128, 136, 2, 128),  # 128
]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,K,N_,n_ids,rank", LONG)
def test_no_row_is_lost(dtype, R, K, N_, n_ids, rank):
    """Sums of whole numbers below 2^24 are exact in any order: a row that is missing or taken twice
    shows.  |v|, |w| <= 4 and at most R rows: sums of at most 4 R < 2^21."""
    s = whole_numbers(dtype, R, K, N_, n_ids, rank, R + rank)
    if dtype == "f32" and R == 9001:
        s["ids"] = s["ids"][torch.randperm(R, generator=torch.Generator().manual_seed(1)).to(DEV)].contiguous()
    o, _ = definition(s["x"], None, s["ids"], s["A"], s["B"], None, s["y"], s["dy"], s["dx"])
    v = moe.moe_adapter_fwd(s["x"], s["ids"], s["A"], s["B"], s["y"], want_v=True)
    r = moe.moe_adapter_bwd(s["dy"], s["x"], s["ids"], s["A"], s["B"], v, s["dx"])
    for n, got in (("v", v), ("y", s["y"]), ("dx", s["dx"]), ("dA", r["dA"]), ("dB", r["dB"])):
        assert torch.equal(got.double(), o[n]), n


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,K,N_,n_ids,rank", LONG[:5])
def test_long_gradients(dtype, R, K, N_, n_ids, rank):
    check(make(dtype, R, K, N_, n_ids, rank, "sorted", False, R + rank))


def test_workspace_of_the_most_rows():
    """Refused where the backward is; below that what R rows need: 4 bytes of the order and 4 of each
    rank value, for 1024 rows two partial sums (rank (K + N) fp32 each) and 16 bytes, and little more."""
    w = L.moe_adapter_ws_bytes
    for rank, dtype, most in ((16, BF16, (1 << 28) - 16), (128, F32, (1 << 30) - 32)):
        for R in (most + 1, (1 << 31) - (1 << 23), 0x7FFF0000):
            assert w(R, 8, 8, 4, rank, dtype) == EUNSUP, (R, rank)
        R = most - 20000
        need = 4 * R * (rank + 1) + R // 512 * rank * 16 * 4 + R // 64
        assert need - (1 << 20) <= w(R, 8, 8, 4, rank, dtype) <= need + (1 << 20)


@gpu
def test_the_most_rows():
    """Near the 2^28 rows of one launch: rows of zeros but for a few at both ends and in the middle,
    whole numbers, forward and backward exact (sums of at most 4 * 300)."""
    R, few = (1 << 28) - 5000, 100
    s = whole_numbers("bf16", 3 * few, 8, 16, 3, 8, 5)
    at = torch.cat([torch.arange(few), torch.arange(few) + R // 2, torch.arange(few) + (R - few)]).to(DEV)
    big = {}
    for n, cols in (("x", 8), ("dy", 16)):
        big[n] = torch.zeros((R, cols), dtype=torch.bfloat16, device=DEV)
        big[n][at] = s[n]
    ids = torch.ones(R, dtype=torch.int32, device=DEV)
    ids[at] = s["ids"]
    y, dx = torch.zeros_like(big["dy"]), torch.zeros_like(big["x"])
    zero = [torch.zeros_like(s[n]) for n in ("y", "dx")]
    o, _ = definition(s["x"], None, s["ids"], s["A"], s["B"], None, zero[0], s["dy"], zero[1])
    v = moe.moe_adapter_fwd(big["x"], ids, s["A"], s["B"], y, want_v=True)
    r = moe.moe_adapter_bwd(big["dy"], big["x"], ids, s["A"], s["B"], v, dx)
    for n, got in (("v", v[at]), ("y", y[at]), ("dx", dx[at]), ("dA", r["dA"]), ("dB", r["dB"])):
        assert torch.equal(got.double(), o[n]), n
    y[at], dx[at] = 0, 0
    assert not y.any() and not dx.any()
