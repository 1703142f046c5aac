"""moe_add_rmsnorm and its backward against their definitions in 64 bits.

The sum is one fp32 addition and one rounding: it matches bit for bit.  A mean square is a sum of
fp32 terms at most 32 + 5 + 16 additions deep, so r is within (53 + 2) / 2 + 2 < 30 half steps
of 2^-24, and the norm, two products later, within 32: 2^-19.  Gradients add a second such
sum over terms of both signs, bounded by the sum of magnitudes: 64 half steps, 2^-18.  bf16
outputs add half a step, 2^-8 of the value.
"""
import numpy as np
import pytest

import few_rows_reference as F

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.float32, torch.bfloat16]
EPS = 1e-6


def data(seed, T, H, dtype, spread=1.0):
    r = np.random.RandomState(seed)
    return torch.from_numpy((r.standard_normal((T, H)) * np.exp(spread * r.standard_normal((T, 1)))).astype(np.float32)).to(dtype)


def gain(seed, H):
    return torch.from_numpy((1 + 0.3 * np.random.RandomState(seed).standard_normal(H)).astype(np.float32))


def f64(t):
    return t.double().cpu().numpy()


def near(got, want, bound):
    got = f64(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


def near8(q, y, n):
    """The codes are within half a step of n, the scale is that of its block, y what the codes stand for."""
    codes, scales = q.codes.view(torch.uint8).cpu().numpy(), q.scales.cpu().numpy()
    v = F.decode8(codes, scales)
    assert np.array_equal(f64(y), v)
    top = F.block_top(n)
    lo, hi = (np.repeat(F.quantize8(n * s)[1], 32, axis=-1) for s in (1 - 2.0 ** -19, 1 + 2.0 ** -19))
    s = np.repeat(scales, 32, axis=-1)
    assert ((lo <= s) & (s <= hi)).all()
    unit = np.ldexp(1.0, s.astype(np.int64) - 127)
    assert (np.abs(v - n) <= np.maximum(2.0 ** -4 * np.abs(n), 2.0 ** -10 * unit) + 2.0 ** -18 * np.abs(n)).all()
    assert (np.abs(v) <= 2 * top).all()


@pytest.mark.parametrize("res", TYPES)
@pytest.mark.parametrize("x", TYPES)
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (5, 31), (1, 32), (9, 64), (17, 1000), (2, 1024), (3, 1025), (4, 1032),
                                 (300, 2021), (2, 3584), (160, 7168), (3, 8200), (2, 16384), (2, 16383)])
def test_forward(T, H, x, res):
    import quantile_balanced_routing_gb300 as Q
    a, b, g = data(T + H, T, H, x), data(T + H + 1, T, H, res, 2.0), gain(H, H)
    got = Q.add_rmsnorm(a.cuda(), g.cuda(), residual=b.cuda(), eps=EPS)
    total = (a.float() + b.float()).to(res)
    assert torch.equal(got.total.cpu(), total) and got.total.dtype == res and got.q is None
    n = F.norm(f64(total), f64(g), EPS)
    assert got.y.dtype == x
    near(got.y, n, (2.0 ** -19 + HALF[x]) * np.abs(n))
    alone = Q.add_rmsnorm(a.cuda(), g.cuda(), eps=EPS)
    n = F.norm(f64(a), f64(g), EPS)
    near(alone.y, n, (2.0 ** -19 + HALF[x]) * np.abs(n))
    assert torch.equal(alone.total.cpu(), a)
    if H % 32 == 0:
        for r, total in ((Q.add_rmsnorm(a.cuda(), g.cuda(), residual=b.cuda(), eps=EPS, mxfp8=True), got.total),
                         (Q.add_rmsnorm(a.cuda(), g.cuda(), eps=EPS, mxfp8=True), a)):
            assert torch.equal(r.total, total.cuda()) and r.y.dtype == torch.bfloat16 and r.q.shape == (T, H)
            near8(r.q, r.y, F.norm(f64(total), f64(g), EPS))
        only = Q.add_rmsnorm(a.cuda(), g.cuda(), eps=EPS, mxfp8=True, values=False)
        assert only.y is None and torch.equal(only.q.codes.view(torch.uint8), r.q.codes.view(torch.uint8))
        assert torch.equal(only.q.scales, r.q.scales)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_in_8_bits_are_exact_at_every_scale(dtype):
    """Rows of +-1 have r = 1, so the norm is the gain itself: all midpoints of the grid, every exponent."""
    import quantile_balanced_routing_gb300 as Q
    mids = np.concatenate([F.E4M3[:120], (F.E4M3[:119] + F.E4M3[1:120]) / 2])
    r = np.random.RandomState(0)
    blocks = []
    for e in list(range(-149, -100)) + list(range(-30, 30)) + list(range(90, 119)):
        m = r.choice(mids, 32) * 2.0
        m[0] = 240.0 if e % 2 else 128.0
        blocks.append(np.ldexp(m * r.choice([-1, 1], 32), e))
    blocks += [np.zeros(32), -np.zeros(32)] + [np.where(np.arange(32) == 5, v, 1.0) for v in (np.inf, -np.inf, np.nan)]
    with np.errstate(over="ignore", under="ignore"):
        g = np.concatenate(blocks).astype(np.float32)
    x = torch.from_numpy(r.choice([-1.0, 1.0], (3, g.size))).to(dtype)
    got = Q.add_rmsnorm(x.cuda(), torch.from_numpy(g).cuda(), eps=0.0, mxfp8=True)
    codes, scales = F.quantize8(f64(x) * g.astype(np.float64))
    assert np.array_equal(got.q.scales.cpu().numpy(), scales)
    assert np.array_equal(got.q.codes.view(torch.uint8).cpu().numpy(), codes)
    v = F.decode8(codes, scales)
    want = torch.from_numpy(v).to(torch.bfloat16)
    assert torch.equal(torch.nan_to_num(got.y.cpu(), nan=7.0), torch.nan_to_num(want, nan=7.0))


@pytest.mark.parametrize("dtotal", [False, True])
@pytest.mark.parametrize("total", TYPES)
@pytest.mark.parametrize("dn", TYPES)
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (1, 32), (9, 64), (70, 1000), (2, 1024), (3, 1025), (77, 3584),
                                 (700, 520), (5, 8200), (650, 2021), (2, 16384), (1300, 40)])
def test_backward(T, H, dn, total, dtotal):
    import quantile_balanced_routing_gb300 as Q
    v, d, o, g = data(T, T, H, total), data(T + 1, T, H, dn), data(T + 2, T, H, total), gain(H, H)
    kw = dict(dtotal=o.cuda()) if dtotal else {}
    dx, dg = Q.add_rmsnorm_backward(d.cuda(), v.cuda(), g.cuda(), eps=EPS, **kw)
    (wx, mx), (wg, mg) = F.norm_backward(f64(d), f64(v), f64(g), f64(o) if dtotal else None, EPS)
    assert dx.dtype == total and dg.dtype == torch.float32
    near(dx, wx, 2.0 ** -18 * mx + HALF[total] * np.abs(wx))
    # a column: its rows a CTA, then 8 warps, 76 parts a run, 8 runs; each term within 2^-19
    near(dg, wg, (2.0 ** -19 + (T + 100) * 2.0 ** -24) * mg)
    again = Q.add_rmsnorm_backward(d.cuda(), v.cuda(), g.cuda(), eps=EPS, **kw)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dg)
    only, none = Q.add_rmsnorm_backward(d.cuda(), v.cuda(), g.cuda(), eps=EPS, need_dgamma=False, **kw)
    assert none is None and torch.equal(only, dx)


def test_strided_rows_and_offset_bases():
    import quantile_balanced_routing_gb300 as Q
    for dtype in TYPES:
        for H, lead, ld in ((64, 0, 96), (64, 1, 97), (1000, 3, 1013), (2048, 8, 2064)):
            wide = data(H, 6, ld, dtype).cuda()
            x, r = wide[:, lead:lead + H], data(H + 1, 6, ld, torch.float32).cuda()[:, lead:lead + H]
            if lead + H > ld:
                continue
            g = torch.cat((torch.zeros(1), gain(H, H))).cuda()[1:].clone() if lead == 0 else gain(H, H).cuda()
            want = Q.add_rmsnorm(x.contiguous(), g, residual=r.contiguous(), mxfp8=H % 32 == 0)
            total = torch.zeros(6, ld, device="cuda")
            got = Q.add_rmsnorm(x, g, residual=r, mxfp8=H % 32 == 0, total=total[:, lead:lead + H])
            assert torch.equal(got.total, want.total) and (total[:, :lead] == 0).all() and (total[:, lead + H:] == 0).all()
            near(got.y, f64(want.y), 2.0 ** -7 * np.abs(f64(want.y)) + 2.0 ** -18)
            dx, dg = Q.add_rmsnorm_backward(x, r, g, dtotal=got.total)
            (wx, mx), (wg, mg) = F.norm_backward(f64(x), f64(r), f64(g), f64(got.total), 1e-6)
            near(dx, wx, 2.0 ** -18 * mx + 2.0 ** -24 * np.abs(wx))
            near(dg, wg, 2.0 ** -17 * mg)


def test_the_residual_stream_in_place_and_leading_axes():
    import quantile_balanced_routing_gb300 as Q
    x, r, g = data(0, 12, 256, torch.bfloat16).cuda(), data(1, 12, 256, torch.bfloat16).cuda(), gain(2, 256).cuda()
    want = Q.add_rmsnorm(x, g, residual=r, mxfp8=True)
    stream = r.clone()
    got = Q.add_rmsnorm(x, g, residual=stream, mxfp8=True, total=stream)
    assert got.total is stream and torch.equal(stream, want.total) and torch.equal(got.y, want.y)
    lead = Q.add_rmsnorm(x.view(3, 4, 256), g, residual=r.view(3, 4, 256), mxfp8=True)
    assert lead.y.shape == (3, 4, 256) and lead.q.scales.shape == (3, 4, 8) and torch.equal(lead.y.view(12, 256), want.y)
    one = Q.add_rmsnorm(x[5], g, residual=r[5])
    assert one.y.shape == (256,) and torch.equal(one.total, want.total[5])


def test_no_rows():
    import quantile_balanced_routing_gb300 as Q
    x, g = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    r = Q.add_rmsnorm(x, g, residual=x, mxfp8=True)
    assert r.y.shape == (0, 64) and r.q.shape == (0, 64)
    dx, dg = Q.add_rmsnorm_backward(x, x, g)
    assert dx.shape == (0, 64) and torch.equal(dg, torch.zeros(64, device="cuda"))


def test_a_bad_row_stays_in_its_row():
    import quantile_balanced_routing_gb300 as Q
    x, g = data(0, 40, 640, torch.float32).cuda(), gain(1, 640).cuda()
    bad = x.clone()
    bad[7, 3], bad[20, 600], bad[30] = float("nan"), float("inf"), 0.0
    a, b = Q.add_rmsnorm(x, g).y, Q.add_rmsnorm(bad, g).y
    ok = torch.ones(40, dtype=torch.bool)
    ok[[7, 20, 30]] = False
    assert torch.equal(a[ok.cuda()], b[ok.cuda()])
    assert torch.isnan(b[7]).all() and torch.isnan(b[20, 600]) and not b[20, :600].any() and not b[30].any()


def test_captured_and_replayed_on_another_stream():
    import quantile_balanced_routing_gb300 as Q
    x, r, g = data(0, 50, 1280, torch.bfloat16).cuda(), data(1, 50, 1280, torch.float32).cuda(), gain(2, 1280).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Q.add_rmsnorm_backward(x, r, g, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = Q.add_rmsnorm(x, g, residual=r, mxfp8=True)
        dx, dg = Q.add_rmsnorm_backward(x, f.total, g, dtotal=f.total)
    x.copy_(data(5, 50, 1280, torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    w = Q.add_rmsnorm(x, g, residual=r, mxfp8=True)
    wx, wg = Q.add_rmsnorm_backward(x, w.total, g, dtotal=w.total)
    assert torch.equal(f.y, w.y) and torch.equal(f.q.scales, w.q.scales) and torch.equal(dx, wx) and torch.equal(dg, wg)


def test_many_short_rows():
    """More rows than a grid dimension of 65535 holds."""
    import quantile_balanced_routing_gb300 as Q
    x, g = data(0, 70000, 32, torch.bfloat16), gain(1, 32)
    n = F.norm(f64(x), f64(g), EPS)
    near(Q.add_rmsnorm(x.cuda(), g.cuda(), eps=EPS).y, n, (2.0 ** -19 + 2.0 ** -8) * np.abs(n))
    wide = x.view(-1, 2240)[:1000].contiguous()
    (wx, mx), (wg, mg) = F.norm_backward(f64(wide), f64(wide), np.ones(2240), None, EPS)
    dx, dg = Q.add_rmsnorm_backward(wide.cuda(), wide.cuda(), torch.ones(2240).cuda(), eps=EPS)
    near(dx, wx, 2.0 ** -18 * mx + 2.0 ** -8 * np.abs(wx))
    near(dg, wg, (2.0 ** -19 + 1100 * 2.0 ** -24) * mg)


@pytest.mark.parametrize("x,res", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("T,H", [(1216, 1032), (1217, 3584), (2500, 1056), (609, 8200), (1531, 8192), (610, 16384),
                                 (1531, 512), (1700, 1032), (3001, 640), (1521, 2048)])
def test_many_rows(T, H, x, res):
    """Rows enough that each CTA takes several in turn."""
    import quantile_balanced_routing_gb300 as Q
    a, b, o, g = data(T, T, H, x), data(T + 1, T, H + 8, res, 2.0)[:, :H], data(T + 2, T, H, res), gain(H, H)
    total = (a.float() + b.float()).to(res)
    n = F.norm(f64(total), f64(g), EPS)
    got = Q.add_rmsnorm(a.cuda(), g.cuda(), residual=b.cuda(), eps=EPS)
    assert torch.equal(got.total.cpu(), total)
    near(got.y, n, (2.0 ** -19 + HALF[x]) * np.abs(n))
    if H % 32 == 0:
        r = Q.add_rmsnorm(a.cuda(), g.cuda(), residual=b.cuda(), eps=EPS, mxfp8=True)
        assert torch.equal(r.total.cpu(), total)
        near8(r.q, r.y, n)
    for dtotal in (None, o):
        kw = {} if dtotal is None else dict(dtotal=o.cuda())
        (wx, mx), (wg, mg) = F.norm_backward(f64(a), f64(total), f64(g), None if dtotal is None else f64(o), EPS)
        dx, dg = Q.add_rmsnorm_backward(a.cuda(), total.cuda(), g.cuda(), eps=EPS, **kw)
        near(dx, wx, 2.0 ** -18 * mx + HALF[res] * np.abs(wx))
        near(dg, wg, (2.0 ** -19 + (T + 100) * 2.0 ** -24) * mg)


@pytest.mark.parametrize("T,H", [(3, 40), (5, 33), (1600, 640)])
def test_gradient_against_differences(T, H):
    """The loss sum(dy n(total)) along random directions of total and gamma, by central differences in 64 bits."""
    import quantile_balanced_routing_gb300 as Q
    v, d, g = data(T, T, H, torch.float32, 0.3), data(T + 1, T, H, torch.float32, 0.3), gain(H, H)
    dx, dg = (f64(t) for t in Q.add_rmsnorm_backward(d.cuda(), v.cuda(), g.cuda(), eps=EPS))
    (_, mx), (_, mg) = F.norm_backward(f64(d), f64(v), f64(g), None, EPS)
    r = np.random.RandomState(H)
    loss = lambda t, c: (f64(d) * F.norm(t, c, EPS)).sum()  # noqa: E731
    h = 1e-5   # the differences' own error: h^2 times the third derivative (at most 100 times the first's sum), and 2^-52 of the loss over h
    for _ in range(4):
        u, c = r.standard_normal((T, H)), r.standard_normal(H)
        got, want = (dx * u).sum(), (loss(f64(v) + h * u, f64(g)) - loss(f64(v) - h * u, f64(g))) / (2 * h)
        noise = 2.0 ** -50 * np.abs(f64(d) * F.norm(f64(v), f64(g), EPS)).sum() / h
        assert abs(got - want) <= ((2.0 ** -18 + 1e-8) * mx * np.abs(u)).sum() + noise
        got, want = (dg * c).sum(), (loss(f64(v), f64(g) + h * c) - loss(f64(v), f64(g) - h * c)) / (2 * h)
        assert abs(got - want) <= ((2.0 ** -19 + (T + 100) * 2.0 ** -24) * mg * np.abs(c)).sum() + noise
