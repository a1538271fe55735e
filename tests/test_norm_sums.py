"""The weights' gradients of the norms over many rows, within a bound that one row left out or added twice
exceeds.

With u = 2^-24.  A gradient is a sum over the rows of dn xh (or dy gate xh).  Its order: a team adds its
rows in a chain, a workgroup its teams, 32 shares the workgroups' partial rows, the first share the others.
The backward has min(ceil(T / 4), 256) workgroups at the least (four teams at the most in one, 256 to 1024
partial rows), so a chain has CHAIN = ceil(T / min(ceil(T / 4), 256)) rows, and with 3 additions of teams,
at most 1024 / 32 = 32 of partial rows and 31 of shares every addend passes through N = CHAIN + 66
roundings.  xh errs by 37 u of itself (36 u of the row's 1 / rms, its product) and, after the layer, by
what c errs: k u s M, M = sum_j |w_j y_j|, and k u rho |xh| through the mean of squares, rho = sum |c| M / sum
c^2; dy gate by 1 u.  So the sum errs by u sum |dn| ((N + 40) |xh| + k (s M + rho |xh|))."""
import math

import numpy as np
import pytest
import torch

import moe_expert_layer_router_amd as moe
from test_norm import DEV, TYPES, U24, close, gather, norm_bwd_ref, norm_ref, rand, routing


def roundings(T):
    return math.ceil(T / min(math.ceil(T / 4), 256)) + 66


def check(got, share, err, what):
    """got [H] against the sum of share [T,H]; err [H] the bound.  The bound is one that sees each row: without
    any one of them most columns are off by more."""
    seen = (share.abs() > 2 * err).double().mean(dim=1)
    assert float(seen.min()) > 0.5, f"{what}: a row is seen in {float(seen.min()):.2f} of the columns"
    close(got, share.sum(dim=0), err, what)


def norm_shares(dn, r, w, eps):
    xh = r * norm_ref(r, w, eps)[1]
    share = dn * xh
    return share, U24 * (roundings(len(r)) + 40) * share.abs().sum(dim=0)


def after_shares(dy, rows, w, gate, eps):
    T, k, H = rows.shape
    c = (rows * w.unsqueeze(2)).sum(dim=1)
    M = (rows.abs() * w.unsqueeze(2)).sum(dim=1)
    s = 1.0 / torch.sqrt((c * c).mean(dim=1, keepdim=True) + eps)
    rho = (c.abs() * M).sum(dim=1, keepdim=True) / (c * c).sum(dim=1, keepdim=True)
    xh = c * s
    share = dy * gate * xh
    err = (dy * gate).abs() * ((roundings(T) + 40) * xh.abs() + k * (s * M + rho * xh.abs()))
    return share, U24 * err.sum(dim=0)


def magnitude(g, *shape, device):
    """Values of both signs between 1/2 and 3/2 in size: every row has a share in every column."""
    v = torch.rand(shape, generator=g, device=device) + 0.5
    return torch.where(torch.rand(shape, generator=g, device=device) < 0.5, -v, v)


def test_bounds_see_a_row():
    """On the CPU: sums without the last row, or with the first one twice, are outside the bound in most
    columns at the largest sizes of the test below; the sums themselves are the formulas'."""
    g = torch.Generator().manual_seed(0)
    T, H, eps = 9000, 64, 1e-5
    r, dn, w = (magnitude(g, *s, device="cpu").double() for s in ((T, H), (T, H), (H,)))
    share, err = norm_shares(dn, r, w, eps)
    assert torch.allclose(share.sum(dim=0), norm_bwd_ref(dn, None, r, w, eps)[1], rtol=0, atol=1e-9)
    for wrong in (share[:-1].sum(dim=0), share.sum(dim=0) + share[0]):
        assert float(((wrong - share.sum(dim=0)).abs() > err).double().mean()) > 0.5
    k = 4
    rows, tw = magnitude(g, T, k, H, device="cpu").double(), torch.rand((T, k), generator=g).double()
    share, err = after_shares(dn, rows, tw, 1.0, eps)
    assert float(((share[:-1].sum(dim=0) - share.sum(dim=0)).abs() > err).double().mean()) > 0.5


NORM = [("bf16", 9000, 64), ("bf16", 4200, 512), ("bf16", 4200, 1024), ("bf16", 4200, 2048), ("bf16", 1300, 4096),
        ("bf16", 600, 8192), ("bf16", 300, 16384), ("f32", 4200, 256), ("f32", 4200, 1024), ("f32", 1300, 2052),
        ("f32", 600, 4096), ("f32", 260, 16384), ("bf16", 7, 512), ("f32", 2, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,T,H", NORM)
def test_norm_weight_gradient_has_every_row_once(dtype, T, H):
    g = torch.Generator(device=DEV).manual_seed(T + H)
    dt, eps = TYPES[dtype], 1e-5
    r, dn = magnitude(g, T, H, device=DEV).to(dt), magnitude(g, T, H, device=DEV).to(dt)
    w = 1.0 + rand(g, H, std=0.2)
    b = moe.moe_norm_bwd(dn, r, w, eps)
    check(b["dweight"], *norm_shares(dn.double().cpu(), r.double().cpu(), w.double().cpu(), eps), "dweight")


AFTER = [(dt, T, H // (1 if dt == "bf16" else 2), k, gate) for dt in ("bf16", "f32")
         for T, H, k, gate in ((9000, 64, 2, "none"), (4200, 512, 8, "token"), (4200, 1024, 1, "full"), (1300, 2048, 7, "full"),
                               (1300, 4096, 4, "none"), (600, 8192, 2, "token"), (270, 16384, 3, "none"), (5, 512, 8, "full"))]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,T,H,k,gate", AFTER)
def test_combine_norm_weight_gradient_has_every_row_once(dtype, T, H, k, gate):
    rng = np.random.default_rng(T + H + k)
    g = torch.Generator(device=DEV).manual_seed(T + k)
    dt, eps = TYPES[dtype], 1e-5
    dest, R = routing(rng, T, k, 1.0)
    assert R == T * k
    y_perm, dy = magnitude(g, R, H, device=DEV).to(dt), magnitude(g, T, H, device=DEV).to(dt)
    tw, w = torch.rand((T, k), generator=g, device=DEV) + 0.1, 1.0 + rand(g, H, std=0.2)
    gt = {"none": None, "token": torch.rand(T, generator=g, device=DEV) + 0.5,
          "full": (torch.rand((T, H), generator=g, device=DEV) + 0.5).to(dt)}[gate]
    b = moe.moe_combine_norm_bwd(dy, y_perm, tw, dest.to(DEV), w, eps, gate=gt)
    gd = 1.0 if gt is None else gt.double().cpu().reshape(T, -1)
    share, err = after_shares(dy.double().cpu(), gather(y_perm.double().cpu(), dest, T, k), tw.double().cpu(), gd, eps)
    check(b["dweight"], share, err, "dweight")
