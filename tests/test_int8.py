"""Rows as 8-bit integers: codes and scales, activation checkpoints, and the int8 products grouped by
expert, against their definitions.

Codes, scales and the values they stand for are defined operation by operation in fp32, so they have to
be equal bit for bit; a product's sum is a whole number, so its result is off by the two scale products
and the conversion (3 u, u = 2^-24) and one rounding to bf16 (2^-8 of the value) of
the exact one.  h = SiLU(g) u: exp(-g) by (2 |g| + 4) u of itself (the argument's product and the
hardware's exponential), 1 / (1 + exp) by another 2 u, two products: (2 |g| + 9) u of h, and its
rounding."""
import numpy as np
import pytest
import torch

from test_abi_cpu import A, BF16, EINVAL, EUNSUP, EWS, F32, L, N, OK, S as STREAM, U, _err
import moe_expert_layer_router_amd as moe

DEV = torch.device("cuda:0")
U24 = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
gpu = pytest.mark.gpu
bf = torch.bfloat16


# ---------------------------------------------------------------------------
# the definitions
# ---------------------------------------------------------------------------

def codes_ref(v, group):
    """v fp32 numpy [rows, cols] -> (codes int8, scales fp32 [rows, cols / group])."""
    b = v.reshape(v.shape[0], -1, group)
    with np.errstate(all="ignore"):
        top = np.abs(b).max(axis=2)
        top = np.where(np.isnan(b).any(axis=2), np.float32("nan"), top).astype(np.float32)
        none = top < np.float32(2.0 ** -100)
        inv = np.where(none, np.float32(0), np.float32(127) / top).astype(np.float32)
        scale = np.where(none, np.float32(0), top / np.float32(127)).astype(np.float32)
        q = np.rint((b * inv[:, :, None]).astype(np.float32))
    return np.nan_to_num(q, nan=0.0).astype(np.int8).reshape(v.shape), scale


def values_ref(q, scale):
    with np.errstate(all="ignore"):
        return (q.reshape(q.shape[0], scale.shape[1], -1).astype(np.float32) * scale[:, :, None]).reshape(q.shape)


def test_definition_of_codes():
    """Worked by hand: largest 127 -> codes are the values, ties to even; largest 254 -> halves."""
    v = np.array([[127, 0.5, 1.5, 2.5, -0.5, -1.5, -127, 3.49] + [0] * 8,
                  [254, 1, 3, 5, -1, -3, -254, 253] + [0] * 8], np.float32)
    q, s = codes_ref(v, 16)
    assert q[0, :8].tolist() == [127, 0, 2, 2, 0, -2, -127, 3] and s[0, 0] == 1
    assert q[1, :8].tolist() == [127, 0, 2, 2, 0, -2, -127, 126] and s[1, 0] == 2
    rng = np.random.default_rng(0)
    v = (rng.standard_normal((64, 96)) * np.exp(rng.uniform(-60, 60, (64, 1)))).astype(np.float32)
    q, s = codes_ref(v, 32)
    err = np.abs(values_ref(q, s).astype(np.float64) - v) / s.repeat(32, axis=1)
    assert err.max() <= 0.5 * (1 + 1e-4)  # half a code, and a code's rounding of 127 u relative
    assert (np.abs(q).reshape(64, 3, 32).max(axis=2) == 127).all()


# ---------------------------------------------------------------------------
# refusals (no GPU)
# ---------------------------------------------------------------------------

def each(f, args, cases):
    for i, v, rc in cases:
        a = list(args)
        a[i] = v
        assert f(*a) == rc, (i, v, _err())


def test_row_refusals():
    q = [A, 8, 64, 32, BF16, N, A, A, STREAM]
    each(L.moe_quantize_i8, q, [(0, N, EINVAL), (0, U, EINVAL), (1, -1, EINVAL), (1, 0x7fffffff, EUNSUP), (2, 0, EINVAL),
                                (2, 72, EINVAL), (3, 0, EINVAL), (3, 48, EINVAL), (3, 16, EUNSUP), (4, 3, EINVAL),
                                (6, N, EINVAL), (6, U, EINVAL), (7, N, EINVAL)])
    assert L.moe_quantize_i8(A, 8, 1920, 320, BF16, N, A, A, STREAM) == EUNSUP and "group" in _err()
    assert L.moe_quantize_i8(A, 1 << 26, 1024, 64, BF16, N, A, A, STREAM) == EUNSUP and "2^32" in _err()
    assert L.moe_quantize_i8(N, 0, 64, 64, F32, N, N, N, STREAM) == OK
    d = [A, A, A, 8, 5, 64, 32, F32, N, A, STREAM]
    each(L.moe_dequantize_i8, d, [(0, N, EINVAL), (1, N, EINVAL), (2, N, EINVAL), (4, -1, EINVAL), (5, 40, EINVAL),
                                  (6, 24, EINVAL), (6, 48, EINVAL), (7, 2, EINVAL), (9, U, EINVAL), (9, N, EINVAL)])
    assert L.moe_dequantize_i8(N, N, N, 0, 0, 64, 64, F32, N, N, STREAM) == OK
    r = [A, A, 8, 64, 32, BF16, N, A, A, STREAM]
    each(L.moe_swiglu_restore_i8, r, [(0, N, EINVAL), (1, N, EINVAL), (2, -1, EINVAL), (3, 0, EINVAL), (3, 24, EINVAL),
                                      (3, 0x40000000, EINVAL), (4, 40, EINVAL), (5, 2, EINVAL), (7, N, EINVAL),
                                      (8, U, EINVAL)])
    assert L.moe_swiglu_restore_i8(N, N, 0, 64, 32, BF16, N, N, N, STREAM) == OK


def test_product_refusals():
    g = [A, A, A, A, 4, 16, 9, 64, 48, A, A, A, STREAM]
    each(L.moe_grouped_gemm_i8, g, [(0, N, EINVAL), (0, U, EINVAL), (1, N, EINVAL), (3, N, EINVAL), (4, 0, EINVAL),
                                    (4, 257, EINVAL), (5, -1, EINVAL), (6, 0, EINVAL), (2, N, EINVAL), (7, 24, EINVAL),
                                    (7, 0, EINVAL), (7, 65552, EUNSUP), (8, 40, EINVAL), (8, (1 << 20) + 16, EUNSUP), (9, U, EINVAL), (10, N, EINVAL),
                                    (10, U, EINVAL), (11, N, EINVAL), (11, U, EINVAL)])
    assert L.moe_grouped_gemm_i8(A, A, A, A, 4, 16, 1 << 20, 2048, 48, A, A, A, STREAM) == EUNSUP and "x_q" in _err()
    assert L.moe_grouped_gemm_i8(A, A, A, A, 4, 16, 9, 65536, 32768, A, A, A, STREAM) == EUNSUP and "weight" in _err()
    assert L.moe_grouped_gemm_i8(A, A, A, A, 256, 0x7fff0000, 9, 16, 1 << 20, A, A, A, STREAM) == EUNSUP and "tiles" in _err()
    assert L.moe_grouped_gemm_i8(N, N, N, N, 4, 0, 0, 64, 48, N, N, N, STREAM) == OK
    f = [A, A, A, A, 4, 16, 9, 64, 48, A, A, A, A, A, A, A, A, A, 1 << 20, STREAM]
    each(L.moe_grouped_ffn_fwd_i8, f, [(i, N, EINVAL) for i in (0, 1, 3, 9, 10, 11, 12, 13, 14, 15, 16)]
         + [(2, N, EINVAL), (4, 0, EINVAL), (7, 40, EINVAL), (8, 40, EINVAL), (7, 65552, EUNSUP), (8, 65552, EUNSUP),
            (17, N, EWS), (17, U, EINVAL), (18, 16, EWS)])
    assert L.moe_grouped_ffn_fwd_i8(A, A, A, A, 4, 1 << 22, 9, 64, 512, A, A, A, A, A, A, A, A, A, 1 << 40, STREAM) == EUNSUP
    assert L.moe_grouped_ffn_fwd_i8(N, N, N, N, 4, 0, 0, 64, 48, N, N, N, N, N, N, N, N, N, 0, STREAM) == OK
    assert L.moe_ffn_i8_ws_bytes(-1, 64) == EINVAL and L.moe_ffn_i8_ws_bytes(4, 20) == EINVAL
    assert L.moe_ffn_i8_ws_bytes(1 << 25, 64) == EUNSUP and L.moe_ffn_i8_ws_bytes(16, 48) >= 16 * 48 + 64


# ---------------------------------------------------------------------------
# rows
# ---------------------------------------------------------------------------

def rows_of(rng, rows, cols, dt):
    v = (rng.standard_normal((rows, cols)) * np.exp(rng.uniform(-20, 20, (rows, 1)))).astype(np.float32)
    return torch.from_numpy(v).to(dt)


ROWS = [(1, 16, None), (5, 48, None), (3, 2048, None), (7, 1040, None), (2, 4096, None), (3, 4112, None), (2, 20000, None),
        (9, 32, 32), (6, 96, 32), (17, 640, 64), (130, 1536, 128), (5, 1024, 256), (3, 1536, 512), (1000, 64, 64)]


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,group", ROWS)
def test_codes_and_values(dtype, rows, cols, group):
    rng = np.random.default_rng(rows + cols)
    dt = TYPES[dtype]
    v = rows_of(rng, rows, cols, dt)
    q, scale = moe.moe_quantize_i8(v.to(DEV), group=group)
    g = group or cols
    want_q, want_s = codes_ref(v.float().numpy(), g)
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(scale.cpu().numpy().reshape(rows, -1), want_s)
    assert scale.shape == ((rows,) if group is None else (rows, cols // group))
    back = moe.moe_dequantize_i8(q, scale, dt)
    assert torch.equal(back.cpu(), torch.from_numpy(values_ref(want_q, want_s)).to(dt))
    src = torch.from_numpy(rng.integers(-2, rows + 2, 2 * rows + 1).astype(np.int32))
    got = moe.moe_dequantize_i8(q, scale, dt, src_row=src.to(DEV)).cpu()
    ok = (src >= 0) & (src < rows)
    assert torch.equal(got[ok], back.cpu()[src[ok].long()]) and (got[~ok] == 0).all()


@gpu
@pytest.mark.parametrize("group", [None, 32])
def test_codes_of_unusual_groups(group):
    cols = 64
    v = torch.zeros((12, cols), dtype=torch.float32)
    v[1, 3] = float("nan")
    v[2, 5], v[2, 6] = float("inf"), 1.0
    v[3, 7] = float("-inf")
    v[4] = 2.0 ** -101
    v[5] = 2.0 ** -100
    v[6] = 3.4e38
    v[7] = 1e-40
    v[8] = torch.arange(64) - 31.5  # ties once scaled by 254 / 127
    v[8, 40] = 127.0
    v[9] = -0.0
    v[10, 0], v[10, 1] = -1.0, 1e-30
    v[11] = torch.linspace(-5, 5, 64)
    q, scale = moe.moe_quantize_i8(v.to(DEV), group=group)
    want_q, want_s = codes_ref(v.numpy(), group or cols)
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(scale.cpu().numpy().reshape(12, -1), want_s, equal_nan=True)
    back = moe.moe_dequantize_i8(q, scale, torch.float32).cpu()
    assert back[1, :32].isnan().all() and back[2, :32].isnan().all() and back[3, :32].isnan().all()
    assert (back[0] == 0).all() and (back[4] == 0).all() and (back[7] == 0).all()
    if group:
        assert (back[1, 32:] == 0).all()  # the next group is not touched


@gpu
def test_rows_past_the_bound_are_left():
    g = torch.Generator(device=DEV).manual_seed(0)
    v = torch.randn((9, 128), generator=g, device=DEV)
    n = torch.tensor([4], dtype=torch.int32, device=DEV)
    for group, shape in ((None, (9,)), (32, (9, 4))):
        q0, s0 = moe.moe_quantize_i8(v, group=group)
        out = {"q": torch.full((9, 128), 7, dtype=torch.int8, device=DEV), "scale": torch.full(shape, 5.0, device=DEV)}
        q, s = moe.moe_quantize_i8(v, group=group, nrows=n, out=out)
        assert torch.equal(q[:4], q0[:4]) and (q[4:] == 7).all() and torch.equal(s[:4], s0[:4]) and (s[4:] == 5).all()
        o = moe.moe_dequantize_i8(q0, s0, bf, nrows=n, out=torch.full((9, 128), 3.0, dtype=bf, device=DEV))
        assert (o[4:] == 3).all() and torch.equal(o[:4], moe.moe_dequantize_i8(q0, s0, bf)[:4])
        r0 = moe.moe_swiglu_restore_i8(q0, s0, bf)
        r = moe.moe_swiglu_restore_i8(q0, s0, bf, nrows=n, out={"gu": torch.full((9, 128), 3.0, dtype=bf, device=DEV),
                                                               "h_perm": torch.full((9, 64), 3.0, dtype=bf, device=DEV)})
        for name in ("gu", "h_perm"):
            assert (r[name][4:] == 3).all() and torch.equal(r[name][:4], r0[name][:4])


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,I,group", [(1, 16, 32), (517, 32, 32), (33, 48, 96), (64, 768, 128), (1, 768, None), (5, 272, 32),
                                          (300, 64, 64)])
def test_restored_gate_up_and_h(dtype, rows, I, group):
    rng = np.random.default_rng(rows + I)
    dt = TYPES[dtype]
    v = torch.from_numpy((rng.standard_normal((rows, 2 * I)) * rng.uniform(0.1, 20, (rows, 1))).astype(np.float32)).to(dt)
    want_q, want_s = codes_ref(v.float().numpy(), group or 2 * I)
    q, s = torch.from_numpy(want_q).to(DEV), torch.from_numpy(want_s).to(DEV)
    r = moe.moe_swiglu_restore_i8(q, s.squeeze(1) if group is None else s, dt)
    gu = torch.from_numpy(values_ref(want_q, want_s)).to(dt)
    assert torch.equal(r["gu"].cpu(), gu)
    g, u = gu[:, :I].double(), gu[:, I:].double()
    h = g * torch.sigmoid(g) * u
    e = torch.finfo(dt).eps / 2
    d = (r["h_perm"].double().cpu() - h).abs()
    assert bool((d <= ((2 * g.abs() + 9) * U24 + e) * h.abs() + 1e-37).all())


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def product_ref(x, xs, src, sizes, w, ws):
    """[R, N] in 64 bits (numpy)."""
    out, lo = [], 0
    for e, n in enumerate(sizes):
        rows = src[lo:lo + n]
        p = x[rows].astype(np.float64) @ w[e].astype(np.float64).T
        out.append(p * xs[rows].astype(np.float64)[:, None] * ws[e].astype(np.float64))
        lo += n
    return np.concatenate(out) if out else np.zeros((0, w.shape[1]))


def off_by(got, want, what):
    d = np.abs(got.double().cpu().numpy() - want)
    bound = (4 * U24 + 2.0 ** -8) * np.abs(want) + 1e-37
    assert (d <= bound).all(), f"{what}: {int((d > bound).sum())} of {d.size}, worst {(d / bound).max():.3g} of its bound"


def product_case(rng, sizes, K, N, x_rows=None, extra=0):
    R = sum(sizes)
    x_rows = x_rows or max(R, 1)
    x = rng.integers(-127, 128, (x_rows, K)).astype(np.int8)
    w = rng.integers(-127, 128, (len(sizes), N, K)).astype(np.int8)
    x[0], w[0, 0] = -128, -128
    xs = rng.uniform(0.5, 2, x_rows).astype(np.float32)
    ws = rng.uniform(0.5, 2, (len(sizes), N)).astype(np.float32)
    src = rng.integers(0, x_rows, R + extra).astype(np.int32)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    return x, xs, src, off, w, ws


def to_gpu(*a):
    return [torch.from_numpy(v).to(DEV) for v in a]


PRODUCTS = [([1], 16, 16), ([1], 2048, 48), ([16], 64, 32), ([17], 48, 80), ([3, 0, 5, 1], 1040, 528), ([0, 0, 33], 80, 16),
            ([64], 128, 128), ([65], 128, 128), ([70, 1, 0, 300], 64, 144), ([256], 192, 128), ([257], 208, 112),
            ([300, 64, 65, 512, 0, 2], 272, 400), ([1] * 256, 32, 32), ([129, 128, 160, 190], 1024, 256),
            ([1000], 768, 2048), ([33] * 16, 512, 272), ([40, 200], 65536, 16), ([600] + [3] * 100, 96, 64),
            # blocks of an expert's rows in several workgroups, more of them than those too
            ([5000], 64, 32), ([300] + [13] * 255, 32, 16), ([0, 64, 0, 65, 128, 1, 129], 2064, 48),
            # large enough for the tiles
            ([256], 192, 4624), ([257], 208, 4624), ([70, 1, 0, 300], 64, 2896), ([300, 64, 65, 512, 0, 2], 272, 2064),
            ([129, 128, 160, 190], 1024, 2064), ([1] * 8 + [400], 1040, 2064), ([33] * 16, 512, 1552),
            ([600] + [3] * 40, 96, 1040), ([1024], 65536, 1280), ([2000] + [0] * 90 + [1], 16, 1040)]


@gpu
@pytest.mark.parametrize("sizes,K,N", PRODUCTS, ids=lambda v: str(v)[:24])
def test_products(sizes, K, N):
    rng = np.random.default_rng(K + N + sum(sizes))
    extra = 5
    x, xs, src, off, w, ws = product_case(rng, sizes, K, N, x_rows=max(3, sum(sizes) // 2), extra=extra)
    R = sum(sizes)
    src[R:] = 1 << 30  # rows past the last group are not read
    dx, dxs, dsrc, doff, dw, dws = to_gpu(x, xs, src, off, w, ws)
    out = torch.full((R + extra, N), 7.0, dtype=bf, device=DEV)
    y = moe.moe_grouped_gemm_i8(dx, dxs, dsrc, doff, dw, dws, out=out)
    assert (y[R:] == 7).all()
    off_by(y[:R], product_ref(x, xs, src, sizes, w, ws), "y")
    # the grouped rows themselves, without a map
    rows = src[:R]
    direct = moe.moe_grouped_gemm_i8(dx[torch.from_numpy(rows.astype(np.int64)).to(DEV)].contiguous(),
                                     dxs[torch.from_numpy(rows.astype(np.int64)).to(DEV)], None, doff, dw, dws)
    assert torch.equal(direct, y[:R])


@gpu
@pytest.mark.parametrize("E,rows", [(3, 5), (1, 400), (256, 4200), (64, 30000)])
def test_no_rows_at_all(E, rows):
    """Every group empty, in both kernels and in the FFN: nothing is written."""
    K, N = 64, 48
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    x, xs = torch.ones((rows, K), dtype=torch.int8, device=DEV), torch.ones(rows, device=DEV)
    w, ws = torch.ones((E, N, K), dtype=torch.int8, device=DEV), torch.ones((E, N), device=DEV)
    d, ds = torch.ones((E, K, N), dtype=torch.int8, device=DEV), torch.ones((E, K), device=DEV)
    y = torch.full((rows, N), 7.0, dtype=bf, device=DEV)
    assert (moe.moe_grouped_gemm_i8(x, xs, None, off, w, ws, out=y) == 7).all()
    o = {"h_perm": y, "y_perm": torch.full((rows, K), 7.0, dtype=bf, device=DEV)}
    moe.moe_grouped_ffn_fwd_i8(x, xs, None, off, (w, ws), (w, ws), (d, ds), out=o)
    assert (y == 7).all() and (o["y_perm"] == 7).all()


@gpu
def test_a_row_that_is_no_number_stays_alone():
    """A token with an infinity and one with a NaN: their rows of the FFN's result are NaN, no other is,
    in both kernels."""
    H, I = 128, 96
    g = torch.Generator(device=DEV).manual_seed(9)
    ww = [moe.moe_quantize_i8(torch.randn(s, generator=g, device=DEV)) for s in ((2, I, H), (2, I, H), (2, H, I))]
    for rows in (12, 150):
        x = torch.randn((rows, H), generator=g, device=DEV).to(bf)
        x[3, 5], x[7, 1] = float("inf"), float("nan")
        off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device=DEV)
        y = moe.moe_grouped_ffn_fwd_i8(*moe.moe_quantize_i8(x), None, off, *ww)["y_perm"]
        bad = y.isnan()
        assert bad[3].all() and bad[7].all() and int(bad.sum()) == 2 * H


@gpu
@pytest.mark.parametrize("N", [208, 1296])
def test_the_split_into_groups_changes_no_bit(N):
    """1030 rows as one group, as groups of 1 to 64 rows beside large ones (tiles for the wider product),
    and as groups that go without tiles."""
    rng = np.random.default_rng(5)
    K, R = 336, 1030
    x, xs, src, _, w, ws = product_case(rng, [R], K, N)
    got = []
    for sizes in ([R], [64, 1, 300, 17, 0, 600, 48], [10] * 103, [R] + [0] * 99):
        off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        E = len(sizes)
        d = to_gpu(x, xs, src, off, np.repeat(w, E, axis=0), np.repeat(ws, E, axis=0))
        got.append(moe.moe_grouped_gemm_i8(*d))
    for y in got[1:]:
        assert torch.equal(y, got[0])


@gpu
@pytest.mark.parametrize("N", [128, 2944])
def test_rows_near_the_end_of_the_address_range(N):
    """2^31 - 2048 bytes of token rows: the last rows through the map, in both kernels."""
    K, x_rows = 2048, (1 << 20) - 1
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randint(-127, 128, (x_rows, K), generator=g, device=DEV, dtype=torch.int8)
    xs = torch.rand(x_rows, generator=g, device=DEV) + 0.5
    w = torch.randint(-127, 128, (2, N, K), generator=g, device=DEV, dtype=torch.int8)
    ws = torch.rand((2, N), generator=g, device=DEV) + 0.5
    src = torch.arange(x_rows - 1, x_rows - 401, -1, device=DEV, dtype=torch.int32)
    off = torch.tensor([0, 350, 400], dtype=torch.int32, device=DEV)
    y = moe.moe_grouped_gemm_i8(x, xs, src, off, w, ws)
    rows = src.cpu().numpy()
    xc, xsc = x[src.long()].cpu().numpy(), xs[src.long()].cpu().numpy()
    want = product_ref(xc, xsc, np.arange(400), [350, 50], w.cpu().numpy(), ws.cpu().numpy())
    off_by(y, want, "y")


FFN = [([2, 0, 1], 64, 48), ([1] * 8, 2048, 768), ([5, 3, 40, 0, 64], 144, 80), ([70, 300, 10], 256, 208),
       ([256, 257, 1, 0], 512, 128), ([64, 65], 16, 16), ([4] * 128, 256, 64), ([256, 257, 1, 0], 2080, 1040),
       # few rows, whose h the down product quantizes itself, in groups of up to 16 and above
       ([1, 2, 0, 1] + [0] * 8, 2048, 768), ([0] * 40 + [37] + [1] * 20, 272, 1024), ([0] * 9 + [5], 64, 16),
       ([1] * 8 + [0] * 8, 64, 1040)]


@gpu
@pytest.mark.parametrize("sizes,H,I", FFN, ids=lambda v: str(v)[:24])
def test_ffn(sizes, H, I):
    """h against the formula; y against the product of the codes of that h, whose rounding to bf16 the
    kernel alone decides where the formula is next to a tie."""
    rng = np.random.default_rng(H + I)
    R, E = sum(sizes), len(sizes)
    x, xs, src, off, wg, gs = product_case(rng, sizes, H, I, x_rows=max(2, R), extra=3)
    xs *= np.float32(1e-4 / H ** 0.5)
    wu, us = rng.integers(-127, 128, wg.shape).astype(np.int8), rng.uniform(0.5, 2, gs.shape).astype(np.float32)
    wd, ds = rng.integers(-127, 128, (E, H, I)).astype(np.int8), rng.uniform(0.5, 2, (E, H)).astype(np.float32)
    src[R:] = -5
    dx, dxs, dsrc, doff, dg, dgs, du, dus, dd, dds = to_gpu(x, xs, src, off, wg, gs, wu, us, wd, ds)
    out = {"h_perm": torch.full((R + 3, I), 7.0, dtype=bf, device=DEV), "y_perm": torch.full((R + 3, H), 7.0, dtype=bf, device=DEV)}
    o = moe.moe_grouped_ffn_fwd_i8(dx, dxs, dsrc, doff, (dg, dgs), (du, dus), (dd, dds), out=out)
    assert (o["h_perm"][R:] == 7).all() and (o["y_perm"][R:] == 7).all()
    g, u = product_ref(x, xs, src, sizes, wg, gs), product_ref(x, xs, src, sizes, wu, us)
    h = g / (1 + np.exp(-g)) * u
    d = np.abs(o["h_perm"][:R].double().cpu().numpy() - h)
    # 3 u of g enter SiLU with a slope of at most 1.1 + its own factor, 3 u of u
    assert (d <= ((2 * np.abs(g) + 9 + 3 + 3 * (1 + np.abs(g))) * U24 + 2.0 ** -8) * np.abs(h) + 1e-37).all()
    hq, hs = codes_ref(o["h_perm"][:R].float().cpu().numpy(), I)
    off_by(o["y_perm"][:R], product_ref(hq, hs[:, 0], np.arange(R), sizes, wd, ds), "y")
    again = moe.moe_grouped_ffn_fwd_i8(dx, dxs, dsrc, doff, (dg, dgs), (du, dus), (dd, dds), ws=o["ws"])
    assert torch.equal(again["y_perm"][:R], o["y_perm"][:R])


@gpu
def test_weights_with_leading_dimensions_and_chain_in_a_graph():
    """Weights quantized as [E,N,K]; quantize, FFN, checkpoint and restore captured in two graphs that are
    replayed in turn over changed inputs, each against the eager bits."""
    g = torch.Generator(device=DEV).manual_seed(1)
    E, H, I, T, k = 6, 128, 96, 50, 2
    ww = [moe.moe_quantize_i8(torch.randn(s, generator=g, device=DEV)) for s in ((E, I, H), (E, I, H), (E, H, I))]
    assert ww[0][0].shape == (E, I, H) and ww[0][1].shape == (E, I)
    flat = moe.moe_quantize_i8(torch.arange(E * 16, device=DEV, dtype=torch.float32).reshape(E, 16))
    assert flat[1].shape == (E,)
    x = torch.randn((T, H), generator=g, device=DEV, dtype=bf)
    gu = torch.randn((T, 2 * I), generator=g, device=DEV, dtype=bf)
    src = torch.randint(0, T, (T * k,), generator=g, device=DEV, dtype=torch.int32)
    off = torch.tensor([0, 30, 30, 61, 70, 71, 98], dtype=torch.int32, device=DEV)

    def chain(keep):
        q, s = moe.moe_quantize_i8(x, out=keep.get("x"))
        f = moe.moe_grouped_ffn_fwd_i8(q, s, src, off, *ww, ws=keep.get("ws"), out=keep.get("f"))
        cq, cs = moe.moe_quantize_i8(gu, group=32, out=keep.get("c"))
        r = moe.moe_swiglu_restore_i8(cq, cs, bf, out=keep.get("r"))
        keep.update(x={"q": q, "scale": s}, f=f, ws=f["ws"], c={"q": cq, "scale": cs}, r=r)
        return f["y_perm"][:98], r["gu"], r["h_perm"]

    stream = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(stream):
        for _ in range(2):
            keep = {}
            chain(keep)
            stream.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                outs = chain(keep)
            graphs.append((graph, outs, keep))
    for _ in range(3):
        x.copy_(torch.randn((T, H), generator=g, device=DEV))
        gu.copy_(torch.randn((T, 2 * I), generator=g, device=DEV))
        eager = chain({})
        torch.cuda.synchronize()
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, outs, _ in graphs:
            for p, q in zip(outs, eager):
                assert torch.equal(p, q)


@gpu
def test_binding_refusals():
    x = torch.zeros((4, 64), device=DEV)
    q, s = moe.moe_quantize_i8(x)
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    w, ws = torch.zeros((1, 32, 64), dtype=torch.int8, device=DEV), torch.ones((1, 32), device=DEV)
    d = (torch.zeros((1, 64, 32), dtype=torch.int8, device=DEV), torch.ones((1, 64), device=DEV))
    src = torch.zeros(4, dtype=torch.int32, device=DEV)
    for bad in (lambda: moe.moe_quantize_i8(x.half()), lambda: moe.moe_quantize_i8(x.t()), lambda: moe.moe_quantize_i8(x[0]),
                lambda: moe.moe_quantize_i8(x, group=48), lambda: moe.moe_quantize_i8(x, group=0), lambda: moe.moe_quantize_i8(x.cpu()),
                lambda: moe.moe_quantize_i8(x, nrows=torch.tensor([1])), lambda: moe.moe_quantize_i8(x, out={"q": q[:2]}),
                lambda: moe.moe_quantize_i8(x, out={"scale": s[:2]}),
                lambda: moe.moe_dequantize_i8(q, s, torch.float16), lambda: moe.moe_dequantize_i8(q, s[:2], bf),
                lambda: moe.moe_dequantize_i8(q.float(), s, bf), lambda: moe.moe_dequantize_i8(q, s.reshape(4, 1).expand(4, 3), bf),
                lambda: moe.moe_dequantize_i8(q, s, bf, src_row=src.long()),
                lambda: moe.moe_swiglu_restore_i8(q, s.double(), bf), lambda: moe.moe_swiglu_restore_i8(q, s, bf, out={"gu": x}),
                lambda: moe.moe_grouped_gemm_i8(q, s[:3], src, off, w, ws), lambda: moe.moe_grouped_gemm_i8(q, s, src, off.long(), w, ws),
                lambda: moe.moe_grouped_gemm_i8(q, s, src, off[:1], w, ws), lambda: moe.moe_grouped_gemm_i8(q, s, src, off, w[:, :, :32], ws),
                lambda: moe.moe_grouped_gemm_i8(q, s, src, off, w[0], ws), lambda: moe.moe_grouped_gemm_i8(q, s, src, off, w, ws[:, :16]),
                lambda: moe.moe_grouped_gemm_i8(q, s, src, off, w, ws, out=x),
                lambda: moe.moe_grouped_ffn_fwd_i8(q, s, src, off, (w, ws), (w, ws), (w, ws)),
                lambda: moe.moe_grouped_ffn_fwd_i8(q, s, src, off, (w, ws), (w.float(), ws), d),
                lambda: moe.moe_grouped_ffn_fwd_i8(q, s, src, off, (w, ws), (w, ws), d, ws=torch.empty(4, device=DEV)),
                lambda: moe.moe_grouped_ffn_fwd_i8(q, s, src, off, (w, ws), (w, ws), d, out={"y_perm": x})):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoEError, match="group"):
        moe.moe_quantize_i8(x, group=16)
