"""Combine with dropout from a counter-based generator (moe_combine_dropout, its backward)
against a float64 definition.  The kept places are those of Philox4x32-10, whose published
test vectors the reference generator here reproduces; they have to be equal bit for bit.

Tolerances (u = 2^-24, e = eps / 2 of the type): y is an fp32 sum of k + 1 terms with a scale,
(k + 4) u times the sum of magnitudes, and one rounding, e |y|; dy_perm two fp32 products and a
rounding; d_topk_w an fp32 sum over H, (H + 4) u times the sum of magnitudes."""
import numpy as np
import pytest
import torch

from test_abi_cpu import A, BF16, EINVAL, F32, L, N, OK, S as STREAM, U, _err
import moe_expert_layer_router_amd as moe

DEV = torch.device("cuda:0")
U24 = 2.0 ** -24
gpu = pytest.mark.gpu


def philox(counter, offset, seed):
    """Words [n, 4] of Philox4x32-10 for an array of 64-bit counters."""
    u, low = np.uint64, np.uint64(0xFFFFFFFF)
    c = [counter & low, counter >> u(32), np.full_like(counter, offset & 0xFFFFFFFF),
         np.full_like(counter, offset >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> u(32)) ^ c[1] ^ u(k0), b & low, (a >> u(32)) ^ c[3] ^ u(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, axis=1)


def keep_mask(seed, offset, T, H, p, t0=0):
    start = t0 * H // 4
    c = np.arange(T * H // 4, dtype=np.uint64) + np.uint64(start)
    return (philox(c, offset, seed) >= np.uint64(int(p * 2 ** 32))).reshape(T, H)


def test_generator_vectors():
    """The three vectors published with the generator (its known answers)."""
    one = lambda c, o, s: [int(v) for v in philox(np.array([c], np.uint64), o, s)[0]]
    full = (1 << 64) - 1
    assert one(0, 0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert one(full, full, full) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert one(0x85A308D3243F6A88, 0x0370734413198A2E, 0x299F31D0A4093822) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_refusals():
    rng = A
    f = L.moe_combine_dropout
    assert f(A, A, A, N, 1.0, rng, 8, 64, 2, F32, A, STREAM) == EINVAL and "[0, 1)" in _err()
    assert f(A, A, A, N, -0.1, rng, 8, 64, 2, F32, A, STREAM) == EINVAL
    assert f(A, A, A, N, float("nan"), rng, 8, 64, 2, F32, A, STREAM) == EINVAL
    assert f(A, A, A, N, 0.1, N, 8, 64, 2, F32, A, STREAM) == EINVAL and "rng" in _err()
    assert f(A, A, A, N, 0.1, U, 8, 64, 2, F32, A, STREAM) == EINVAL and "8-byte" in _err()
    assert f(N, A, A, N, 0.1, rng, 8, 64, 2, F32, A, STREAM) == EINVAL and "y_perm" in _err()
    assert f(A, A, N, N, 0.1, rng, 8, 64, 2, F32, A, STREAM) == EINVAL and "dest_row" in _err()
    assert f(A, A, A, U, 0.1, rng, 8, 64, 2, F32, A, STREAM) == EINVAL and "residual" in _err()
    assert f(A, A, A, N, 0.1, rng, 8, 64, 2, F32, U, STREAM) == EINVAL
    assert f(A, A, A, N, 0.1, rng, 8, 66, 2, F32, A, STREAM) == EINVAL
    assert f(A, A, A, N, 0.1, rng, 8, 68, 2, BF16, A, STREAM) == EINVAL
    assert f(A, A, A, N, 0.1, rng, 8, 64, 33, F32, A, STREAM) == EINVAL
    assert f(A, A, A, N, 0.1, rng, -8, 64, 2, F32, A, STREAM) == EINVAL
    assert f(A, A, A, N, 0.1, rng, 2 ** 31 - 1, 64, 1, F32, A, STREAM) == -2
    assert f(A, A, A, N, 0.1, rng, 8, 64, 2, 7, A, STREAM) == EINVAL
    assert f(N, N, N, N, 0.1, N, 0, 64, 2, F32, N, STREAM) == OK
    g = L.moe_combine_dropout_bwd
    assert g(A, A, A, A, 1.5, rng, 8, 64, 2, F32, A, A, STREAM) == EINVAL
    for i, name in ((0, "dy"), (1, "y_perm"), (2, "topk_w"), (3, "dest_row"), (10, "dy_perm"), (11, "d_topk_w")):
        a = [A, A, A, A, 0.1, rng, 8, 64, 2, F32, A, A, STREAM]
        a[i] = N
        assert g(*a) == EINVAL and name in _err()
    assert g(N, N, N, N, 0.1, N, 0, 64, 2, F32, N, N, STREAM) == OK


def routing(rng, T, k, local):
    """dest_row of a permutation over a random part `local` of the slots, and its row count."""
    slots = rng.random(T * k) < local
    R = int(slots.sum())
    dest = np.full(T * k, -1, np.int32)
    dest[slots] = rng.permutation(R)
    return dest, R


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


CASES = [  # dtype, T, H, k, share of local slots, p, residual
    ("bf16", 1, 8, 1, 1.0, 0.5, True), ("f32", 1, 4, 1, 1.0, 0.5, False), ("bf16", 5, 64, 2, 0.5, 0.0, True),
    ("f32", 257, 60, 3, 0.7, 0.3, True), ("bf16", 130, 520, 8, 1.0, 0.1, True),
    ("bf16", 33, 2048, 8, 0.12, 0.25, False), ("f32", 19, 2052, 8, 1.0, 0.9, True),
    ("bf16", 7, 4104, 32, 1.0, 0.999, True), ("bf16", 64, 768, 5, 0.0, 0.1, True),
    ("f32", 64, 768, 5, 0.0, 0.1, False),
]


@gpu
@pytest.mark.parametrize("dtype,T,H,k,local,p,with_res", CASES)
def test_against_definition(dtype, T, H, k, local, p, with_res):
    rng = np.random.default_rng(T * 7 + H)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    e = torch.finfo(dt).eps / 2 if dtype == "bf16" else U24
    dest, R = routing(rng, T, k, local)
    rows = T * k + 3
    y_perm = dev(rng.standard_normal((rows, H)), dt)
    y_perm[R:] = float("nan")  # rows in use by nobody are never read
    w = dev(rng.random((T, k)).astype(np.float32))
    res = dev(rng.standard_normal((T, H)), dt) if with_res else None
    dy = dev(rng.standard_normal((T, H)), dt)
    seed, offset = 0x9123456789ABCDEF, (1 << 40) + T
    state = torch.tensor([seed - (1 << 64), offset], dtype=torch.int64, device=DEV)
    keep = keep_mask(seed, offset, T, H, p)
    scale = 1.0 / (1.0 - p)
    yp, wh = y_perm.double().cpu().numpy(), w.double().cpu().numpy()
    local_slots = (dest >= 0).reshape(T, k)
    picked = np.where(local_slots[..., None], yp[np.maximum(dest, 0)].reshape(T, k, H), 0.0)
    ref = scale * keep * (wh[..., None] * picked).sum(axis=1)
    mag = scale * keep * (wh[..., None] * np.abs(picked)).sum(axis=1)
    if with_res:
        ref = ref + res.double().cpu().numpy()
        mag = mag + np.abs(res.double().cpu().numpy())
    y = moe.moe_combine_dropout(y_perm, w, dev(dest), T, p, state, residual=res)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= (k + 4) * U24 * mag * (1 + e) + e * np.abs(ref)).all(), err.max()

    out = {"dy_perm": torch.full((rows, H), float("nan"), dtype=dt, device=DEV)}
    b = moe.moe_combine_dropout_bwd(dy, y_perm, w, dev(dest), p, state, out=out)
    g = scale * keep * dy.double().cpu().numpy()
    got = b["dy_perm"].double().cpu().numpy()
    assert np.isnan(got[R:]).all(), "rows behind the last were written"
    t_of = np.repeat(np.arange(T), k)[dest >= 0]
    ref_d = np.zeros((R, H))
    ref_d[dest[dest >= 0]] = wh.reshape(-1)[dest >= 0][:, None] * g[t_of]
    assert (np.abs(got[:R] - ref_d) <= (e + 4 * U24) * np.abs(ref_d)).all()
    ref_w = (picked * g[:, None]).sum(axis=2)
    mag_w = (np.abs(picked) * np.abs(g)[:, None]).sum(axis=2)
    assert (np.abs(b["d_topk_w"].cpu().numpy() - ref_w) <= (H + 4) * U24 * mag_w).all()
    if local == 0.0:
        assert not b["d_topk_w"].any()


@gpu
def test_gradient_against_differences():
    """The backward is the derivative of the forward: <dy, y(w + h) - y(w - h)> / 2h, fp32."""
    rng = np.random.default_rng(2)
    T, H, k, p = 6, 32, 3, 0.4
    dest, R = routing(rng, T, k, 0.8)
    yp, w = dev(rng.standard_normal((R, H)).astype(np.float32)), rng.random((T, k)).astype(np.float32)
    dy = rng.standard_normal((T, H)).astype(np.float32)
    state = torch.tensor([11, 12], dtype=torch.int64, device=DEV)
    b = moe.moe_combine_dropout_bwd(dev(dy), yp, dev(w), dev(dest), p, state)
    f = lambda w, yp: (moe.moe_combine_dropout(yp, dev(w), dev(dest), T, p, state).double().cpu().numpy() * dy).sum()
    h = 2.0 ** -4  # y is linear in w and in y_perm: no error of the step, that of y's rounding over h
    for t in range(T):
        for j in range(k):
            d = np.zeros_like(w)
            d[t, j] = h
            num = (f(w + d, yp) - f(w - d, yp)) / (2 * h)
            assert abs(num - float(b["d_topk_w"][t, j])) <= 64 * H * U24 / h * 8
    for r, c in ((0, 0), (R - 1, H - 1), (R // 2, 5)):
        d = torch.zeros_like(yp)
        d[r, c] = h
        num = (f(w, yp + d) - f(w, yp - d)) / (2 * h)
        assert abs(num - float(b["dy_perm"][r, c])) <= 64 * H * U24 / h * 8


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropped_elements_hide_infinities(dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T, H, p, seed, offset = 9, 256, 0.5, 3, 4
    keep = torch.from_numpy(keep_mask(seed, offset, T, H, p)).to(DEV)
    state = torch.tensor([seed, offset], dtype=torch.int64, device=DEV)
    dest = torch.arange(T, dtype=torch.int32, device=DEV)
    w = torch.ones(T, 1, device=DEV)
    yp = torch.where(keep, 1.0, float("inf")).to(dt)
    yp[3] = torch.where(keep[3], 1.0, float("nan")).to(dt)
    res = torch.full((T, H), 0.5, dtype=dt, device=DEV)
    y = moe.moe_combine_dropout(yp, w, dest, T, p, state, residual=res, out=res)
    assert torch.equal(y, torch.where(keep, 2.5, 0.5).to(dt))  # in place of the residual
    b = moe.moe_combine_dropout_bwd(torch.ones_like(yp), yp, w, dest, p, state)
    assert torch.equal(b["dy_perm"], torch.where(keep, 2.0, 0.0).to(dt))
    assert torch.equal(b["d_topk_w"][:, 0], 2.0 * keep.sum(dim=1))


@gpu
def test_counters_past_32_bits():
    """2^34 elements: the counter of the last rows does not fit 32 bits, their bytes lie past 2^35."""
    H, p, seed, offset = 2048, 0.5, 77, 5
    T = (1 << 23) + 3
    dest = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    dest[-4:] = torch.arange(4, dtype=torch.int32, device=DEV)
    yp = torch.ones(4, H, dtype=torch.bfloat16, device=DEV)
    state = torch.tensor([seed, offset], dtype=torch.int64, device=DEV)
    y = moe.moe_combine_dropout(yp, None, dest, T, p, state)
    keep = torch.from_numpy(keep_mask(seed, offset, 4, H, p, t0=T - 4)).to(DEV)
    assert torch.equal(y[-4:], torch.where(keep, 2.0, 0.0).bfloat16())
    assert not y[:4].any() and not y[T // 2:T // 2 + 4].any()


@gpu
def test_captured_with_numbers_advanced_between_replays():
    rng = np.random.default_rng(1)
    T, H, k, p = 300, 512, 4, 0.2
    dest, R = routing(rng, T, k, 0.6)
    dest = dev(dest)
    yp, dy = dev(rng.standard_normal((T * k, H)), torch.bfloat16), dev(rng.standard_normal((T, H)), torch.bfloat16)
    w = dev(rng.random((T, k)).astype(np.float32))
    state = torch.tensor([5, 0], dtype=torch.int64, device=DEV)
    y = moe.moe_combine_dropout(yp, w, dest, T, p, state)
    b = moe.moe_combine_dropout_bwd(dy, yp, w, dest, p, state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_combine_dropout(yp, w, dest, T, p, state, out=y)
        moe.moe_combine_dropout_bwd(dy, yp, w, dest, p, state, out=b)
        state[1] += 1
    seen = []
    side = torch.cuda.Stream()
    for i in range(4):
        before = state.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert int(state[1]) == i + 1
        with torch.cuda.stream(side):
            ye = moe.moe_combine_dropout(yp, w, dest, T, p, before)
            be = moe.moe_combine_dropout_bwd(dy, yp, w, dest, p, before)
        side.synchronize()
        assert torch.equal(ye, y) and torch.equal(be["dy_perm"][:R], b["dy_perm"][:R])
        assert torch.equal(be["d_topk_w"], b["d_topk_w"])
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1])


@gpu
def test_binding_refusals():
    yp, w = torch.zeros(8, 16, device=DEV), torch.ones(4, 2, device=DEV)
    dest, state = torch.arange(8, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int64, device=DEV)
    a = dict(y_perm=yp, topk_w=w, dest_row=dest, T=4, p=0.1, rng=state)
    for bad in (dict(y_perm=yp.half()), dict(topk_w=w.double()), dict(topk_w=w[:3]), dict(T=3), dict(T=-1),
                dict(rng=state.int()), dict(rng=state.cpu()), dict(residual=torch.zeros(4, 16).to(DEV).bfloat16()),
                dict(out=torch.zeros(4, 8, device=DEV)), dict(dest_row=dest.long())):
        with pytest.raises(ValueError):
            moe.moe_combine_dropout(**{**a, **bad})
    with pytest.raises(moe.MoEError, match="p="):
        moe.moe_combine_dropout(**{**a, "p": 1.0})
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_combine_dropout(yp.cpu(), w, dest, 4, 0.1, state)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_binding_refusals_of_whole_calls(dtype):
    """Calls that give every tensor: as they are they pass, with any one tensor of another type, shape,
    device or order they are refused."""
    rand = lambda *s: torch.randn(*s, device=DEV).to(dtype)
    a = dict(y_perm=rand(8, 16), topk_w=torch.rand(4, 2, device=DEV),
             dest_row=torch.arange(8, dtype=torch.int32, device=DEV), T=4, p=0.1,
             rng=torch.tensor([3, 5], device=DEV), residual=rand(4, 16), out=rand(4, 16))
    want = moe.moe_combine_dropout(**{**a, "out": None})
    assert moe.moe_combine_dropout(**a) is a["out"] and torch.equal(a["out"], want)
    b = {n: a[n] for n in ("y_perm", "topk_w", "dest_row", "p", "rng")}
    b.update(dy=rand(4, 16), out=dict(dy_perm=rand(8, 16), d_topk_w=torch.zeros(4, 2, device=DEV)))
    fresh = moe.moe_combine_dropout_bwd(**{**b, "out": None})
    got = moe.moe_combine_dropout_bwd(**b)
    assert all(got[n] is b["out"][n] and torch.equal(got[n], fresh[n]) for n in b["out"])

    def bad(t):
        yield t.cpu()
        yield t.double()
        if t is not a["y_perm"]:  # (whose row count no other tensor gives)
            yield t[1:]
        if t.numel() > 1:  # (one element is dense at any stride)
            yield torch.stack([t, t], -1)[..., 0]
        yield t.unsqueeze(0)

    for call, args in ((moe.moe_combine_dropout, a), (moe.moe_combine_dropout_bwd, b)):
        for name, t in args.items():
            if torch.is_tensor(t):
                for u in bad(t):
                    with pytest.raises(ValueError):
                        call(**{**args, name: u})
    for name, t in b["out"].items():
        for u in bad(t):
            with pytest.raises(ValueError):
                moe.moe_combine_dropout_bwd(**{**b, "out": {**b["out"], name: u}})


def test_sizes_past_one_launch_are_refused():
    """A launch has fewer than 2^32 threads, 64 for a token."""
    T = (1 << 26) - 3
    assert L.moe_combine_dropout(A, A, A, N, 0.1, A, T, 8, 1, BF16, A, STREAM) == -2 and "2^32" in _err()
    assert L.moe_combine_dropout_bwd(A, A, A, A, 0.1, A, T, 8, 1, BF16, A, A, STREAM) == -2 and "2^32" in _err()


@gpu
def test_the_most_tokens():
    """2^26 - 4 tokens, a wave for each: the last ones' elements lie past 2^29."""
    H, p, seed, offset = 8, 0.5, 21, 9
    T = (1 << 26) - 4
    dest = torch.arange(T, dtype=torch.int32, device=DEV)
    yp = torch.ones(T, H, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(T, 1, device=DEV)
    state = torch.tensor([seed, offset], dtype=torch.int64, device=DEV)
    y = moe.moe_combine_dropout(yp, w, dest, T, p, state)
    b = moe.moe_combine_dropout_bwd(yp, yp, w, dest, p, state)
    for t0 in (0, T // 2, T - 500):
        keep = torch.from_numpy(keep_mask(seed, offset, 500, H, p, t0=t0)).to(DEV)
        want = torch.where(keep, 2.0, 0.0).bfloat16()
        assert torch.equal(y[t0:t0 + 500], want) and torch.equal(b["dy_perm"][t0:t0 + 500], want)
        assert torch.equal(b["d_topk_w"][t0:t0 + 500, 0], want.float().sum(dim=1))
