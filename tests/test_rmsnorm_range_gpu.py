"""The norm and its gradient of rows whose squares, or whose products with the gradient, leave fp32's range.

The normed row does not depend on the row's size where eps is 0 or far below its mean square: the tolerances are those
of ordinary rows, 2^-19 for the norm and 2^-18 of the sum of magnitudes for the gradients, the output's rounding, and
half of fp32's least number, 2^-150 (2^-134 for bf16).
"""
import numpy as np
import pytest

import few_rows_reference as F

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
LEAST = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134}
TYPES = [torch.float32, torch.bfloat16]
# one row or a few, odd widths, a warp and a CTA a row, rows in a ring (two and four pieces a thread)
SIZES = [(3, 7), (9, 64), (5, 1000), (2, 1025), (4, 3584), (3, 16384), (3100, 512), (1300, 1056), (400, 7168), (310, 8448)]


def f64(t):
    return t.double().cpu().numpy()


def near(got, want, bound):
    got = f64(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


def rows(r, T, H, dtype, power):
    """Rows of about 2^power, each a little larger or smaller."""
    x = r.standard_normal((T, H)) * np.exp(0.3 * r.standard_normal((T, 1))) + r.choice([-0.5, 0.5], (T, 1))
    return torch.from_numpy(np.ldexp(x, power).clip(-3e38, 3e38)).to(dtype)


def gain(r, H):
    return torch.from_numpy((1 + 0.3 * r.standard_normal(H)).astype(np.float32))


@pytest.mark.parametrize("power", [-120, -78, -52, -40, 40, 62, 66, 100, 124])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H", SIZES)
def test_forward(T, H, dtype, power):
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(T + H + power + 200)
    x, b, g = rows(r, T, H, dtype, power), rows(r, T, H, dtype, power), gain(r, H)
    for eps in (0.0, 1e-30, 1e-6):
        n = F.norm(f64(x), f64(g), float(np.float32(eps)))
        near(Q.add_rmsnorm(x.cuda(), g.cuda(), eps=eps).y, n, (2.0 ** -19 + HALF[dtype]) * np.abs(n) + LEAST[dtype])
    total = (x.float() + b.float()).to(dtype)
    n = F.norm(f64(total), f64(g), 0.0)
    got = Q.add_rmsnorm(x.cuda(), g.cuda(), residual=b.cuda(), eps=0.0)
    assert torch.equal(got.total.cpu(), total)
    near(got.y, n, (2.0 ** -19 + HALF[dtype]) * np.abs(n) + LEAST[dtype])
    if H % 32 == 0:
        got = Q.add_rmsnorm(x.cuda(), g.cuda(), residual=b.cuda(), eps=0.0, mxfp8=True)
        v = F.decode8(got.q.codes.view(torch.uint8).cpu().numpy(), got.q.scales.cpu().numpy())
        assert np.array_equal(f64(got.y), v)
        assert (np.abs(v - n) <= (2.0 ** -4 + 2.0 ** -18) * np.abs(n) + 2.0 ** -17 * F.block_top(n)).all()


@pytest.mark.parametrize("power", [-120, -78, -52, -40, 40, 62, 66, 100, 124])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H", SIZES)
def test_backward(T, H, dtype, power):
    """The gradient dn as large as the rows, so that dx is of the gain's size."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(T + H + power + 200)
    v, d, o, g = rows(r, T, H, dtype, power), rows(r, T, H, dtype, min(power, 100)), rows(r, T, H, dtype, 0), gain(r, H)
    for eps, dtotal in ((0.0, None), (0.0, o), (1e-30, None), (1e-6, o)):
        if eps == 1e-6 and power < 0:
            continue   # (dx is then what dtotal is)
        kw = {} if dtotal is None else dict(dtotal=o.cuda())
        (wx, mx), (wg, mg) = F.norm_backward(f64(d), f64(v), f64(g), None if dtotal is None else f64(o), float(np.float32(eps)))
        dx, dg = Q.add_rmsnorm_backward(d.cuda(), v.cuda(), g.cuda(), eps=eps, **kw)
        # dn gamma and the mean of its products with the normed row are fp32 numbers, half of the least one off where they are
        # that small; dx takes them times 1 / rms, the mean times the normed row as well
        v64 = f64(v)
        inverse = F.rms(v64, float(np.float32(eps)))
        small = 2.0 ** -149 * inverse * (1 + np.abs(v64) * inverse)
        near(dx, wx, 2.0 ** -18 * mx + HALF[dtype] * np.abs(wx) + LEAST[dtype] + small)
        near(dg, wg, (2.0 ** -19 + (T + 100) * 2.0 ** -24) * mg + T * LEAST[torch.float32])


@pytest.mark.parametrize("H", [64, 1025, 4096])
def test_a_large_gradient_of_ordinary_rows(H):
    """dn gamma total passes fp32's range, the gradient does not."""
    import quantile_balanced_routing_gb300 as Q
    for T in (5, 1000):
        r = np.random.RandomState(H + T)
        v, d, g = rows(r, T, H, torch.float32, 20), rows(r, T, H, torch.float32, 112), gain(r, H)
        for total in (v, v.to(torch.bfloat16)):
            dx, dg = Q.add_rmsnorm_backward(d.cuda(), total.cuda(), g.cuda(), eps=1e-6)
            (wx, mx), (wg, mg) = F.norm_backward(f64(d), f64(total), f64(g), None, 1e-6)
            near(dx, wx, 2.0 ** -18 * mx + HALF[total.dtype] * np.abs(wx))
            near(dg, wg, (2.0 ** -19 + (T + 100) * 2.0 ** -24) * mg)


@pytest.mark.parametrize("T,H", SIZES)
def test_rows_beside_them_stay(T, H):
    """Rows of every size, of zeros, infinities and NaN between ordinary ones, whose bits do not change."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(T + H)
    x, d, g = rows(r, T, H, torch.bfloat16, 0), rows(r, T, H, torch.bfloat16, -10), gain(r, H).cuda()
    bad = x.clone()
    at = np.arange(0, T, 3)
    bad[at] = (x[at].double() * torch.from_numpy(np.ldexp(1.0, r.choice([-120, -70, 62, 120], (len(at), 1))))).to(torch.bfloat16)
    bad[at[0], 0] = float("inf")
    if len(at) > 2:
        bad[at[1]], bad[at[2], -1] = 0.0, float("nan")
    keep = np.setdiff1d(np.arange(T), at)
    a, b = Q.add_rmsnorm(x.cuda(), g).y, Q.add_rmsnorm(bad.cuda(), g).y
    assert torch.equal(a[keep], b[keep]) and torch.isnan(b[at[0], 0]) and not b[at[0], 1:].any()
    if len(at) > 2:
        assert not b[at[1]].any() and torch.isnan(b[at[2]]).all()
    a, b = Q.add_rmsnorm_backward(d.cuda(), x.cuda(), g)[0], Q.add_rmsnorm_backward(d.cuda(), bad.cuda(), g)[0]
    assert torch.equal(a[keep], b[keep])
