"""RMS norms around the layer (moe_norm, moe_combine_norm and their backwards) against the formulas in
64 bits.

Tolerances, with u = 2^-24 (half a step of fp32) and e = eps / 2 of the stored type:
 - a row's sum is a chain of at most 32 products in a lane, 6 levels over the wave and up to 16
   waves: it errs by at most 60 u times the sum of magnitudes, which for squares is the sum itself, so
   s = 1 / sqrt(mean + eps) by 30 u + 4 u (division, addition, square root, reciprocal) of itself: S = 36 u;
 - c is a chain of k products: k u M, M = sum_j |w_j y_j|; through the mean of squares that is another
   k u rho of s, rho = sum |c| M / sum c^2;
 - a sum over T rows errs by at most (T + 70) u times the sum of magnitudes (rows of a workgroup in a
   chain, then at most 64 partial rows a share and 32 shares);
 - every stored value by e of itself.
Second-order terms (below 1e-3 of these) are covered by rounding each count up."""
import numpy as np
import pytest
import torch

from test_abi_cpu import A, BF16, EINVAL, EUNSUP, EWS, F32, L, N, OK, S as STREAM, U, _err
import moe_expert_layer_router_amd as moe

DEV = torch.device("cuda:0")
U24 = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
gpu = pytest.mark.gpu


def half_step(dt):
    return torch.finfo(dt).eps / 2


# ---------------------------------------------------------------------------
# the formulas in 64 bits
# ---------------------------------------------------------------------------

def norm_ref(r, weight, eps):
    s = 1.0 / torch.sqrt((r * r).mean(dim=1, keepdim=True) + eps)
    return r * s * weight, s


def norm_bwd_ref(dn, dr, r, weight, eps):
    _, s = norm_ref(r, weight, eps)
    xh, g = r * s, dn * weight
    dx = s * (g - xh * (g * xh).mean(dim=1, keepdim=True))
    return dx + (0 if dr is None else dr), (dn * xh).sum(dim=0)


def gather(y_perm, dest, T, k):
    rows = torch.zeros((T * k, y_perm.shape[1]), dtype=torch.float64)
    local = dest >= 0
    rows[local] = y_perm[dest[local].long()]
    return rows.reshape(T, k, -1)


def after_ref(rows, w, residual, rs, gate, weight, eps):
    """rows [T,k,H] (0 for non-local slots), gate [T,1], [T,H] or 1."""
    c = (rows * w.unsqueeze(2)).sum(dim=1)
    s = 1.0 / torch.sqrt((c * c).mean(dim=1, keepdim=True) + eps)
    return rs * residual + gate * (c * s) * weight, c, s


def after_bwd_ref(dy, rows, w, gate, weight, eps):
    c = (rows * w.unsqueeze(2)).sum(dim=1)
    s = 1.0 / torch.sqrt((c * c).mean(dim=1, keepdim=True) + eps)
    xh, g = c * s, dy * gate * weight
    dc = s * (g - xh * (g * xh).mean(dim=1, keepdim=True))
    return dict(dc=dc, dw=(rows * dc.unsqueeze(1)).sum(dim=2), dweight=(dy * gate * xh).sum(dim=0),
                dgate=dy * weight * xh)


def test_formulas_against_autograd_and_differences():
    g = torch.Generator().manual_seed(3)
    T, k, H, eps = 5, 3, 12, 1e-3
    R = lambda *s: torch.randn(s, generator=g, dtype=torch.float64).requires_grad_()
    x, delta, weight, dn, dr = R(T, H), R(T, H), R(H), R(T, H), R(T, H)

    def loss1(x, delta, weight):
        r = x + delta
        return (norm_ref(r, weight, eps)[0] * dn).sum() + (r * dr).sum()

    got = torch.autograd.grad(loss1(x, delta, weight), (x, delta, weight))
    dx, dweight = norm_bwd_ref(dn, dr, x + delta, weight, eps)
    for a, b in zip(got, (dx, dx, dweight)):
        assert torch.allclose(a, b, rtol=0, atol=1e-12)
    rows, w, gate, res, dy = R(T, k, H), R(T, k), R(T, H), R(T, H), R(T, H)

    def loss2(rows, w, gate, weight, res):
        return (after_ref(rows, w, res, 0.5, gate, weight, eps)[0] * dy).sum()

    args = [rows, w, gate, weight, res]
    got = torch.autograd.grad(loss2(*args), args)
    f = after_bwd_ref(dy, rows, w, gate, weight, eps)
    want = (w.unsqueeze(2) * f["dc"].unsqueeze(1), f["dw"], f["dgate"], f["dweight"], 0.5 * dy)
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=0, atol=1e-11)
    with torch.no_grad():  # central differences, error of the order h^2 = 1e-10 times third derivatives
        h = 1e-5
        for i, a in enumerate(args):
            v = torch.randn(a.shape, generator=g, dtype=torch.float64)
            up = loss2(*[t + h * v if j == i else t for j, t in enumerate(args)])
            dn_ = loss2(*[t - h * v if j == i else t for j, t in enumerate(args)])
            assert abs(float((up - dn_) / (2 * h) - (want[i] * v).sum())) < 1e-5


# ---------------------------------------------------------------------------
# refusals (no GPU)
# ---------------------------------------------------------------------------

def test_norm_refusals():
    f = L.moe_norm
    assert f(A, A, A, 1e-6, 8, 64, 7, A, A, STREAM) == EINVAL and "dtype" in _err()
    assert f(A, A, A, 1e-6, -1, 64, F32, A, A, STREAM) == EINVAL and "T" in _err()
    assert f(A, A, A, 1e-6, 8, 66, F32, A, A, STREAM) == EINVAL
    assert f(A, A, A, 1e-6, 8, 60, BF16, A, A, STREAM) == EINVAL
    assert f(A, A, A, 1e-6, 8, 0, F32, A, A, STREAM) == EINVAL
    assert f(A, A, A, 1e-6, 8, 16392, BF16, A, A, STREAM) == EUNSUP and "16384" in _err()
    for eps in (0.0, -1.0, float("nan"), float("inf"), 1e-46, 1e300):
        assert f(A, A, A, eps, 8, 64, F32, A, A, STREAM) == EINVAL and "eps" in _err()
    assert f(A, A, A, 1e-6, 0x7fffffff, 64, F32, A, A, STREAM) == EUNSUP
    assert f(A, A, A, 1e-6, 1 << 26, 64, F32, A, A, STREAM) == EUNSUP and "2^32" in _err()
    assert f(A, A, A, 1e-6, 1 << 22, 16384, BF16, A, A, STREAM) == EUNSUP and "2^32" in _err()
    for i, name in ((0, "x"), (1, "delta"), (2, "weight"), (7, "r"), (8, "n")):
        a = [A, A, A, 1e-6, 8, 64, F32, A, A, STREAM]
        a[i] = U
        assert (f(*a) == EINVAL and "16-byte" in _err()), name
        a[i] = N
        assert i == 1 or (f(*a) == EINVAL and name in _err())
    assert f(N, N, N, 1e-6, 0, 64, F32, N, N, STREAM) == OK
    b = L.moe_norm_bwd
    args = lambda: [A, A, 1.0, A, A, 1e-6, 8, 64, F32, A, A, 0, A, 1 << 30, STREAM]
    for i, name in ((0, "dn"), (3, "r"), (4, "weight"), (9, "dx"), (10, "dweight")):
        a = args()
        a[i] = N
        assert b(*a) == EINVAL and name in _err()
    for i, v, rc in ((1, U, EINVAL), (11, 2, EINVAL), (12, N, EWS), (12, U, EINVAL), (13, 64, EWS), (7, 16400, EUNSUP)):
        a = args()
        a[i] = v
        assert b(*a) == rc, i
    assert L.moe_norm_ws_bytes(0) == EINVAL and L.moe_norm_ws_bytes(16385) == EUNSUP
    assert L.moe_norm_ws_bytes(16384) > 0


def test_combine_norm_refusals():
    f = L.moe_combine_norm
    args = lambda: [A, A, A, A, 1.0, A, 1, A, 1e-6, 8, 64, 2, F32, A, STREAM]
    for i, name in ((0, "y_perm"), (2, "dest_row"), (5, "gate"), (7, "weight"), (13, "y ")):
        a = args()
        a[i] = N
        assert f(*a) == EINVAL and name in _err()
    for i, v, rc in ((0, U, EINVAL), (3, U, EINVAL), (6, 3, EINVAL), (6, -1, EINVAL), (7, U, EINVAL), (8, 0.0, EINVAL),
                     (9, -1, EINVAL), (10, 65, EINVAL), (10, 16388, EUNSUP), (11, 0, EINVAL), (11, 33, EINVAL),
                     (12, 5, EINVAL), (13, U, EINVAL), (9, 1 << 26, EUNSUP)):
        a = args()
        a[i] = v
        assert f(*a) == rc, (i, v)
    a = args()
    a[5], a[6] = U, 2
    assert f(*a) == EINVAL and "gate" in _err()
    assert f(N, N, N, N, 1.0, N, 0, N, 1e-6, 0, 64, 2, F32, N, STREAM) == OK
    b = L.moe_combine_norm_bwd
    args = lambda: [A, A, A, A, A, 1, A, 1e-6, 8, 64, 2, F32, A, A, A, A, 0, A, 1 << 30, STREAM]
    for i, name in ((0, "dy"), (1, "y_perm"), (2, "topk_w"), (3, "dest_row"), (4, "gate"), (6, "weight"),
                    (12, "dy_perm"), (13, "d_topk_w"), (14, "dgate"), (15, "dweight")):
        a = args()
        a[i] = N
        assert b(*a) == EINVAL and name in _err()
    for i, v, rc in ((16, 3, EINVAL), (17, N, EWS), (18, 100, EWS), (10, 40, EINVAL), (5, 9, EINVAL)):
        a = args()
        a[i] = v
        assert b(*a) == rc, (i, v)


# ---------------------------------------------------------------------------
# the kernels
# ---------------------------------------------------------------------------

def close(got, want, bound, what):
    d = (got.double().cpu() - want).abs()
    bad = ~(d <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float((d / bound)[bad].max()):.3g} of its bound"


def rand(g, *shape, std=1.0, dt=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dt)


NORM = [("bf16", 1, 2048), ("bf16", 3, 8), ("bf16", 130, 512), ("bf16", 129, 1024), ("bf16", 65, 1032),
        ("bf16", 2051, 2048), ("bf16", 37, 2056), ("bf16", 9, 8192), ("bf16", 5, 16384), ("f32", 1, 4),
        ("f32", 77, 64), ("f32", 1003, 516), ("f32", 33, 1024), ("f32", 33, 2052), ("f32", 7, 4096),
        ("f32", 4, 16384), ("bf16", 9000, 64)]
# more rows than one a team of the backward, in every shape
NORM += [(dt, T, H // (1 if dt == "bf16" else 2)) for dt in ("bf16", "f32")
         for T, H in ((4200, 512), (4200, 1024), (4200, 2048), (600, 4096), (300, 8192), (270, 9008))]
NORM += [("f32", 260, 9008), ("f32", 260, 16384)]


@gpu
@pytest.mark.parametrize("dtype,T,H", NORM)
@pytest.mark.parametrize("parts", ["both", "none"])
def test_norm_against_formula(dtype, T, H, parts):
    g = torch.Generator(device=DEV).manual_seed(T * 31 + H)
    dt, eps = TYPES[dtype], 1e-5
    e = half_step(dt)
    both = parts == "both"
    x, weight, dn = rand(g, T, H, std=2.0, dt=dt), 1.0 + rand(g, H, std=0.2), rand(g, T, H, dt=dt)
    delta, dr = (rand(g, T, H, dt=dt), rand(g, T, H, dt=dt)) if both else (None, None)
    f = moe.moe_norm(x, weight, eps, delta=delta)
    rs = 0.625
    b = moe.moe_norm_bwd(dn, f["r"], weight, eps, dr=dr, dr_scale=rs)
    want_r = (x.float() + delta.float()).to(dt) if both else x
    assert torch.equal(f["r"], want_r)
    r, w = want_r.double().cpu(), weight.double().cpu()
    n, s = norm_ref(r, w, eps)
    close(f["n"], n, (40 * U24 + e) * n.abs() + 1e-37, "n")
    dnd, drd = dn.double().cpu(), (rs * dr.double().cpu() if both else None)
    dx, dw = norm_bwd_ref(dnd, drd, r, w, eps)
    xh, gg = (r * s).abs(), (dnd * w).abs()
    size = s * (gg + xh * (gg * xh).mean(dim=1, keepdim=True))  # s twice in the mean, once outside, and the sum: below 150 u
    size = 150 * size + (2 * drd.abs() if both else 0)
    close(b["dx"], dx, U24 * size + (2 * U24 + e) * dx.abs() + 1e-37, "dx")
    close(b["dweight"], dw, (T + 120) * U24 * (dnd * r * s).abs().sum(dim=0) + 1e-37, "dweight")


def routing(rng, T, k, local):
    """dest_row of a permutation over a random part `local` of the slots, and its row count."""
    slots = rng.random(T * k) < local
    R = int(slots.sum())
    dest = np.full(T * k, -1, np.int32)
    dest[slots] = rng.permutation(R)
    return torch.from_numpy(dest), R


AFTER = [("bf16", 1, 2048, 8, "none", 1.0), ("bf16", 33, 2048, 8, "full", 1.0), ("bf16", 517, 2048, 8, "token", 1.0),
         ("bf16", 40, 512, 3, "token", 0.5), ("bf16", 41, 8, 1, "none", 0.7), ("bf16", 35, 1024, 9, "full", 0.9),
         ("bf16", 21, 768, 32, "token", 1.0), ("bf16", 1500, 64, 2, "full", 0.6), ("bf16", 11, 4096, 8, "token", 0.8),
         ("bf16", 6, 8192, 10, "full", 1.0), ("bf16", 4, 16384, 4, "token", 1.0), ("bf16", 5, 16384, 17, "none", 0.4),
         ("f32", 256, 64, 2, "token", 1.0), ("f32", 19, 516, 6, "full", 0.8), ("f32", 23, 1024, 8, "none", 1.0),
         ("f32", 9, 2052, 20, "full", 0.9), ("f32", 5, 16384, 3, "token", 1.0), ("f32", 13, 260, 5, "none", 0.0),
         ("bf16", 3000, 2048, 2, "token", 0.6)]
# every shape of a row's waves with one to eight slots held, more tokens than one a team of the backward
AFTER += [(dt, T, H // (1 if dt == "bf16" else 2), k, gate, 0.8) for dt in ("bf16", "f32")
          for T, H in ((4200, 512), (2100, 1024), (1100, 2048), (560, 4096), (300, 8192), (270, 9008))
          for k, gate in ((1, "full"), (4, "none"), (7, "token"))]
AFTER += [("f32", 260, 9008, 2, "none", 0.8), ("f32", 260, 8192, 3, "token", 0.8), ("f32", 260, 16384, 4, "full", 0.9)]


@gpu
@pytest.mark.parametrize("dtype,T,H,k,gate,local", AFTER)
def test_combine_norm_against_formula(dtype, T, H, k, gate, local):
    rng = np.random.default_rng(T * 7 + H + k)
    g = torch.Generator(device=DEV).manual_seed(T + H)
    dt, eps, rs = TYPES[dtype], 1e-5, 0.625
    e = half_step(dt)
    dest, R = routing(rng, T, k, local)
    y_perm = torch.full((T * k, H), float("nan"), dtype=dt, device=DEV)  # rows past R are never read
    y_perm[:R] = rand(g, R, H, dt=dt)
    w = torch.softmax(rand(g, T, k), dim=1)
    weight, residual, dy = 1.0 + rand(g, H, std=0.2), rand(g, T, H, dt=dt), rand(g, T, H, dt=dt)
    gt = {"none": None, "token": torch.sigmoid(rand(g, T)), "full": torch.sigmoid(rand(g, T, H)).to(dt)}[gate]
    dest_d = dest.to(DEV)
    y = moe.moe_combine_norm(y_perm, w, dest_d, T, weight, eps, residual=residual, residual_scale=rs, gate=gt)
    guard = torch.full((T * k, H), 7.0, dtype=dt, device=DEV)
    b = moe.moe_combine_norm_bwd(dy, y_perm, w, dest_d, weight, eps, gate=gt, out={"dy_perm": guard})
    assert (b["dy_perm"][R:] == 7.0).all()
    # definitions
    wd, weightd, dyd, resd = (t.double().cpu() for t in (w, weight, dy, residual))
    gd = 1.0 if gt is None else gt.double().cpu().reshape(T, -1)
    rows = gather(y_perm.double().cpu(), dest, T, k)
    want, c, s = after_ref(rows, wd, resd, rs, gd, weightd, eps)
    f = after_bwd_ref(dyd, rows, wd, gd, weightd, eps)
    # error magnitudes, in units of u
    M = (rows.abs() * wd.unsqueeze(2)).sum(dim=1)
    rho = ((c.abs() * M).sum(dim=1, keepdim=True) / (c * c).sum(dim=1, keepdim=True)).nan_to_num(0.0, 0.0, 0.0)
    xh, es = c * s, k * rho + 36
    exh = k * s * M + (es + 1) * xh.abs()
    tiny = 1e-37
    gw = (gd * weightd).abs()
    close(y, want, U24 * (gw * (exh + 3 * xh.abs()) + 3 * (rs * resd).abs()) + (2 * U24 + e) * want.abs() + tiny, "y")
    gg = (dyd * gd * weightd)
    m = (gg * xh).mean(dim=1, keepdim=True)
    em = (gg.abs() * (exh + 64 * xh.abs())).mean(dim=1, keepdim=True)
    edc = s * (4 * gg.abs() + exh * m.abs() + xh.abs() * em + 4 * (xh * m).abs()) + (es + 2) * f["dc"].abs()
    local_slot = (dest >= 0).reshape(T, k)
    ydp = torch.zeros((T * k, H), dtype=torch.float64)
    bound = torch.full((T * k, H), 1.0, dtype=torch.float64)
    to = dest[dest >= 0].long()
    v = (wd.unsqueeze(2) * f["dc"].unsqueeze(1)).reshape(T * k, H)[dest >= 0]
    ydp[to] = v
    bound[to] = U24 * (wd.unsqueeze(2) * edc.unsqueeze(1)).reshape(T * k, H)[dest >= 0] + (2 * U24 + e) * v.abs() + tiny
    close(b["dy_perm"][:R], ydp[:R], bound[:R], "dy_perm")
    edw = (rows.abs() * (edc + 64 * f["dc"].abs()).unsqueeze(1)).sum(dim=2)
    close(b["d_topk_w"], torch.where(local_slot, f["dw"], 0.0), U24 * edw + tiny, "d_topk_w")
    size = (dyd * gd).abs()
    close(b["dweight"], f["dweight"],
          U24 * (size * exh + (T + 72) * (size * xh.abs())).sum(dim=0) + tiny, "dweight")
    full = (dyd * weightd).abs()
    if gate == "token":
        close(b["dgate"], f["dgate"].sum(dim=1), U24 * (full * (exh + 66 * xh.abs())).sum(dim=1) + tiny, "dgate")
    elif gate == "full":
        close(b["dgate"], f["dgate"], U24 * full * (exh + 4 * xh.abs()) + e * f["dgate"].abs() + tiny, "dgate")
    else:
        assert b["dgate"] is None


@gpu
def test_no_slots_no_residual_and_weights_of_one():
    """Tokens whose slots are all elsewhere: residual_scale * residual, and 0 without one; topk_w None."""
    T, H, k = 4, 128, 2
    g = torch.Generator(device=DEV).manual_seed(1)
    y_perm, weight = rand(g, T * k, H), torch.ones(H, device=DEV)
    dest = torch.tensor([-1, -1, 1, 0, -1, 2, -1, -1], dtype=torch.int32, device=DEV)
    res = rand(g, T, H)
    y = moe.moe_combine_norm(y_perm, None, dest, T, weight, 1e-6, residual=res, residual_scale=2.0)
    assert torch.equal(y[0], 2 * res[0]) and torch.equal(y[3], 2 * res[3])
    c = torch.stack([y_perm[1].double() + y_perm[0].double(), y_perm[2].double()])
    want = 2 * res[1:3].double() + c / torch.sqrt((c * c).mean(dim=1, keepdim=True) + 1e-6)
    assert float((y[1:3].double() - want).abs().max()) < 60 * U24 * 8  # values below 8
    y = moe.moe_combine_norm(y_perm, None, dest, T, weight, 1e-6)
    assert (y[0] == 0).all() and (y[3] == 0).all()


@gpu
def test_rows_of_zeros_and_of_one_token_and_nan_stays_in_its_row():
    H = 256
    x = torch.zeros((3, H), device=DEV)
    x[1] = float("nan")
    x[2] = 3.0
    w = torch.ones(H, device=DEV)
    f = moe.moe_norm(x, w, 1e-6)
    assert (f["n"][0] == 0).all() and f["n"][1].isnan().all()
    assert float((f["n"][2].double() - 3.0 / (9.0 + 1e-6) ** 0.5).abs().max()) < 40 * U24
    b = moe.moe_norm_bwd(torch.ones_like(x), x, w, 1e-6)
    assert b["dx"][1].isnan().all() and torch.isfinite(b["dx"][[0, 2]]).all()
    assert float((b["dx"][0].double() - 1e3).abs().max()) < 150 * U24 * 1e3  # s = 1 / sqrt(eps)


@gpu
def test_in_place_accumulate_and_no_rows():
    g = torch.Generator(device=DEV).manual_seed(2)
    T, H = 40, 512
    x, delta, dn, dr = (rand(g, T, H, dt=torch.bfloat16) for _ in range(4))
    w = rand(g, H)
    f = moe.moe_norm(x, w, delta=delta)
    b = moe.moe_norm_bwd(dn, f["r"], w, dr=dr)
    x2, n2 = x.clone(), torch.empty_like(x)
    f2 = moe.moe_norm(x2, w, delta=delta, out={"r": x2, "n": n2})
    assert torch.equal(x2, f["r"]) and torch.equal(f2["n"], f["n"])
    dr2, dw2 = dr.clone(), b["dweight"].clone()
    b2 = moe.moe_norm_bwd(dn, f["r"], w, dr=dr2, accumulate=True, ws=b["ws"], out={"dx": dr2, "dweight": dw2})
    assert torch.equal(dr2, b["dx"]) and torch.equal(dw2, b["dweight"] + b["dweight"])
    dn2 = dn.clone()
    moe.moe_norm_bwd(dn2, f["r"], w, dr=dr, out={"dx": dn2})
    assert torch.equal(dn2, b["dx"])
    none = x[:0]
    assert moe.moe_norm(none, w, delta=none)["n"].shape == (0, H)
    e = moe.moe_norm_bwd(none, none, w, out={"dweight": dw2})
    assert (dw2 == 0).all() and e["dx"].shape == (0, H)
    e = moe.moe_norm_bwd(none, none, w, accumulate=True, out={"dweight": torch.full((H,), 3.0, device=DEV)})
    assert (e["dweight"] == 3).all()
    i32 = torch.zeros(0, dtype=torch.int32, device=DEV)
    k = torch.zeros((0, 2), device=DEV)
    assert moe.moe_combine_norm(none, k, i32, 0, w).shape == (0, H)
    e = moe.moe_combine_norm_bwd(none, none, k, i32, w)
    assert (e["dweight"] == 0).all()


@gpu
@pytest.mark.parametrize("gate", ["none", "token", "full"])
def test_captured_and_replayed_on_another_stream(gate):
    """Forward and backward of both norms in one graph, replayed over changed inputs, with eager work
    and another graph's replays between; each replay has the eager result's bits."""
    g = torch.Generator(device=DEV).manual_seed(4)
    T, H, k, dt = 300, 1024, 4, torch.bfloat16
    rng = np.random.default_rng(0)
    dest, R = routing(rng, T, k, 0.9)
    dest = dest.to(DEV)
    a = dict(x=rand(g, T, H, dt=dt), delta=rand(g, T, H, dt=dt), y_perm=rand(g, T * k, H, dt=dt), dy=rand(g, T, H, dt=dt))
    w, weight = torch.softmax(rand(g, T, k), dim=1), rand(g, H)
    gt = {"none": None, "token": rand(g, T), "full": rand(g, T, H, dt=dt)}[gate]

    def step(keep):
        f = moe.moe_norm(a["x"], weight, delta=a["delta"], out=keep.get("f"))
        y = moe.moe_combine_norm(a["y_perm"], w, dest, T, weight, residual=f["n"], residual_scale=0.5, gate=gt,
                                 out=keep.get("y"))
        b = moe.moe_combine_norm_bwd(a["dy"], a["y_perm"], w, dest, weight, gate=gt, ws=keep.get("ws"),
                                     out=keep.get("b") or {"dy_perm": torch.zeros_like(a["y_perm"])})
        d = moe.moe_norm_bwd(a["dy"], f["r"], weight, dr=y, ws=b["ws"], out=keep.get("d"))
        keep.update(f=f, y=y, b=b, d=d, ws=b["ws"])
        outs = [f["n"], f["r"], y, b["dy_perm"], b["d_topk_w"], b["dweight"], d["dx"], d["dweight"]]
        return outs + ([] if gt is None else [b["dgate"]])

    stream = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(stream):
        for _ in range(2):
            keep = {}
            step(keep)
            stream.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                outs = step(keep)
            graphs.append((graph, outs, keep))
    for i in range(3):
        for n in a:
            a[n].copy_(rand(g, *a[n].shape, dt=dt))
        eager = step({})
        torch.cuda.synchronize()
        for graph, outs, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, outs, _ in graphs:
            for p, q in zip(outs, eager):
                assert torch.equal(p, q)


@gpu
def test_binding_refusals():
    x, w = torch.zeros((4, 64), device=DEV), torch.ones(64, device=DEV)
    for bad in (lambda: moe.moe_norm(x.cpu(), w), lambda: moe.moe_norm(x, w[:32]), lambda: moe.moe_norm(x, w.bfloat16()),
                lambda: moe.moe_norm(x.half(), w), lambda: moe.moe_norm(x.t(), w), lambda: moe.moe_norm(x[0], w),
                lambda: moe.moe_norm(x, w, delta=x[:2]), lambda: moe.moe_norm(x, w, delta=x.bfloat16()),
                lambda: moe.moe_norm(x, w, out={"n": x[:2]}), lambda: moe.moe_norm_bwd(x, x[:2], w),
                lambda: moe.moe_norm_bwd(x, x, w, accumulate=True),
                lambda: moe.moe_norm_bwd(x, x, w, ws=torch.empty(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    dest, tw = torch.zeros(8, dtype=torch.int32, device=DEV), torch.zeros((4, 2), device=DEV)
    yp = torch.zeros((8, 64), device=DEV)
    ok = dict(y_perm=yp, topk_w=tw, dest_row=dest, T=4, weight=w)
    for n, v in (("y_perm", yp.half()), ("topk_w", tw[:2]), ("dest_row", dest[:6]), ("dest_row", dest.long()), ("T", 3),
                 ("weight", w[:8]), ("residual", x[:2]), ("gate", tw), ("gate", w[:3]), ("gate", x[:, :32]),
                 ("gate", x.unsqueeze(0)), ("out", x[:2])):
        with pytest.raises(ValueError):
            moe.moe_combine_norm(**{**ok, n: v})
    with pytest.raises(ValueError):
        moe.moe_combine_norm(**{**ok, "topk_w": None, "dest_row": dest[:7]})
    ok = dict(dy=x, y_perm=yp, topk_w=tw, dest_row=dest, weight=w)
    for n, v in (("dy", x[:2]), ("y_perm", yp[:, :32]), ("topk_w", tw.double()), ("gate", w), ("accumulate", True),
                 ("out", {"dgate": x, "dweight": w[:8]})):
        with pytest.raises(ValueError):
            moe.moe_combine_norm_bwd(**{**ok, n: v})
    with pytest.raises(moe.MoEError, match="eps"):
        moe.moe_norm(x, w, eps=0.0)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [64, 520, 1024, 2048, 3000, 4096, 8192, 9000])
def test_a_token_has_the_same_bits_among_few_and_many(H, dtype):
    dt, T, k, few = TYPES[dtype], 1100, 3, 37
    g = torch.Generator(device=DEV).manual_seed(H)
    yp = torch.randn((T * k, H), generator=g, device=DEV).to(dt)
    tw = torch.rand((T, k), generator=g, device=DEV)
    dest = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32)
    dest[1::7] = -1
    w = torch.rand(H, generator=g, device=DEV) + 0.5
    y = moe.moe_combine_norm(yp, tw, dest, T, w)
    for t0 in (0, T - few):
        part = moe.moe_combine_norm(yp, tw[t0:t0 + few], dest[t0 * k:(t0 + few) * k].contiguous(), few, w)
        assert torch.equal(y[t0:t0 + few], part)
