"""moe_mxfp4_* against their definitions in 64 bits.

Quantisation is a whole-number result: codes, scales and values match bit for
bit.  Products of E2M1 values times powers of two are exact in fp32, so a
product differs from the exact sum by the fp32 additions, at most
(terms) 2^-24 of the sum of magnitudes, and by the one rounding of the output:
2^-8 of its value covers bf16.
"""
import numpy as np
import pytest

import mx_reference as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def rows(r, R, K, spread=1.0):
    x = r.standard_normal((R, K)) * np.exp(spread * r.standard_normal((R, 1)))
    return torch.from_numpy(x.astype(np.float32))


def near(got, want, mags, terms, bf16):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    bound = terms * 2.0 ** -24 * mags + (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(want)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 96), (257, 544), (64, 7168), (5000, 64)])
def test_quantize_exact(R, K, dtype):
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(R + K)
    x = rows(r, R, K, 3.0)
    x[::3, ::5] = 0.0
    x[:, -1] = torch.from_numpy(r.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.99], R).astype(np.float32))
    x[R // 2, :32] = 0.0
    x = x.to(getattr(torch, dtype))
    q, v = Q.mxfp4_quantize(x.cuda(), values=True)
    codes, scales, values = M.quantize(x.double().numpy())
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert v.dtype == x.dtype and np.array_equal(v.double().cpu().numpy(), values)
    only = Q.mxfp4_quantize(x.cuda())
    assert torch.equal(only.codes, q.codes) and torch.equal(only.scales, q.scales)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantize_every_tie_and_every_scale(dtype):
    """All midpoints of the grid at every block exponent, from the smallest subnormals to the largest numbers."""
    import quantile_balanced_routing_gb300 as Q
    steps = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7])
    block = np.concatenate([steps, -steps])
    x = np.stack([np.ldexp(block, e - 2) for e in range(-148, 128)])
    x = torch.from_numpy(x.astype(np.float32)).to(getattr(torch, dtype))
    q, v = Q.mxfp4_quantize(x.cuda(), values=True)
    codes, scales, values = M.quantize(x.double().numpy())
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(v.double().cpu().numpy(), values)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_quantize_marks_blocks_that_are_not_finite(bad):
    import quantile_balanced_routing_gb300 as Q
    x = torch.ones(4, 96)
    x[2, 40] = bad
    q, v = Q.mxfp4_quantize(x.cuda(), values=True)
    s = q.scales.cpu()
    assert s[2, 1] == 255 and (s != 255).sum() == 11
    assert torch.isnan(v[2, 32:64]).all() and torch.isnan(v).sum() == 32
    assert not q.codes[2, 16:32].any()


def test_quantize_strided_rows_and_leading_axes():
    import quantile_balanced_routing_gb300 as Q
    x = rows(np.random.RandomState(5), 33, 128)
    want = Q.mxfp4_quantize(x.cuda())
    wide = torch.full((33, 192), float("nan")).cuda()
    wide[:, 64:] = x.cuda()
    got = Q.mxfp4_quantize(wide[:, 64:])
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    three = Q.mxfp4_quantize(x.view(3, 11, 128).cuda())
    assert three.shape == (3, 11, 128) and torch.equal(three.codes.view(33, 64), want.codes)
    empty = Q.mxfp4_quantize(x[:0].cuda())
    assert empty.shape == (0, 128)


def test_quantized_weights_run_in_the_layer():
    """The codes are what the layer takes: an MXFP4 layer on weights quantised here against one on their values."""
    import quantile_balanced_routing_gb300 as Q
    torch.manual_seed(3)
    d, L, n, k, m, T = 512, 512, 16, 2, 512, 32
    g = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    dense = dict(w_router=g(n, d) / d ** .5, w_down=g(L, d) / d ** .5, w_proj_up=g(d, L) / L ** .5)
    dense = {a: b.bfloat16() for a, b in dense.items()}
    dense["rms_gamma"] = torch.ones(L, device="cuda")
    w = {a: Q.mxfp4_quantize((g(n, r, c) / c ** .5).bfloat16(), values=True)
         for a, r, c in (("gate", m, L), ("up", m, L), ("out", L, m))}
    x = g(T, d).bfloat16()
    outs = []
    for fmt in ("mxfp4", "bf16"):
        lay = Q.LatentMoE(d, L, n, k, m, 0, expert_wfmt=fmt, max_tokens=T)
        t = dict(dense)
        for a, (q, v) in w.items():
            t["w_" + a] = q.codes if fmt == "mxfp4" else v
            if fmt == "mxfp4":
                t["s_" + a] = q.scales
        lay.set_weights(**t)
        outs.append(lay.forward(x).float())
        assert lay.status() == 0
        lay.close()
    a, b = outs
    err = (a - b).abs().amax(1) / b.abs().amax(1)
    assert float(err.max()) < 2e-2        # the layer's own bf16 tolerance


# ---------------------------------------------------------------------- product

PRODUCTS = [
    # R, E (0: one matrix), N, K, skew
    (1, 0, 8, 32, 0.0),
    (1, 0, 136, 544, 0.0),
    (5, 0, 264, 96, 0.0),
    (17, 0, 128, 256, 0.0),
    (130, 0, 256, 1056, 0.0),
    (300, 0, 520, 320, 0.0),
    (1, 3, 64, 64, 0.0),
    (40, 7, 72, 160, 3.0),          # experts without rows
    (611, 24, 264, 544, 2.0),
    (900, 2, 384, 288, 0.2),
    (513, 64, 128, 1024, 0.5),
    (2, 1000, 16, 32, 0.0),
    (1500, 3, 136, 2080, 0.1),
    (2100, 0, 1288, 800, 0.0),
]


def product_case(R, E, N, K, skew):
    r = np.random.RandomState(R * 7 + E + N + K)
    xq = M.quantize(rows(r, R, K).numpy())
    wq = M.quantize((rows(r, max(1, E) * N, K, 0.3) / K ** 0.5).numpy())
    offsets = None
    if E:
        p = np.exp(skew * r.standard_normal(E))
        offsets = np.concatenate([[0], np.cumsum(r.multinomial(R, p / p.sum()))]).astype(np.int32)
    dy = torch.from_numpy(r.standard_normal((R, N)).astype(np.float32)).bfloat16()
    return xq, wq, offsets, dy


def on_gpu(Q, xq, wq, offsets, E, N, K):
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    lead = (E, N) if E else (N,)
    return (Q.Mxfp4(t(xq[0]), t(xq[1])), Q.Mxfp4(t(wq[0]).view(*lead, K // 2), t(wq[1]).view(*lead, K // 32)),
            None if offsets is None else t(offsets))


@pytest.mark.parametrize("R,E,N,K,skew", PRODUCTS)
def test_product(R, E, N, K, skew):
    import quantile_balanced_routing_gb300 as Q
    xq, wq, offsets, _ = product_case(R, E, N, K, skew)
    y = Q.mxfp4_matmul(*on_gpu(Q, xq, wq, offsets, E, N, K))
    want, mags = M.matmul(xq[2], wq[2].reshape(max(1, E), N, K), offsets)
    assert y.dtype == torch.bfloat16
    near(y, want, mags, K, True)
    assert Q.qbmoe_status(None, None) == 0


@pytest.mark.parametrize("dw_dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("R,E,N,K,skew", PRODUCTS)
def test_product_gradients(R, E, N, K, skew, dw_dtype):
    import quantile_balanced_routing_gb300 as Q
    xq, wq, offsets, dy = product_case(R, E, N, K, skew)
    x, w, off = on_gpu(Q, xq, wq, offsets, E, N, K)
    dx, dw = Q.mxfp4_matmul_backward(dy.cuda(), x, w, off, dw_dtype=getattr(torch, dw_dtype))
    (wx, mx), (ww, mw) = M.matmul_backward(dy.double().numpy(), xq[2], wq[2].reshape(max(1, E), N, K), offsets)
    near(dx, wx, mx, N, True)
    near(dw.view(max(1, E), N, K), ww, mw, R, dw_dtype == "bfloat16")
    assert Q.qbmoe_status(None, None) == 0


@pytest.mark.parametrize("R,E,N,K", [(20000, 1, 136, 96), (30011, 3, 64, 160), (9000, 1, 2048, 2560), (13000, 2, 1032, 2304)])
def test_weight_gradient_over_many_rows(R, E, N, K):
    """Long sums, in parts (few tiles) and in segments (many): an fp32 gradient keeps the accuracy of fp32 additions.
    A sum of R products with random signs is within about sqrt(R) 2^-24 of its size when each addition rounds;
    the tensor cores' own accumulation over R rows would be off by R 2^-32 or so, ten times that at these sizes."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(R)
    xq = M.quantize(rows(r, R, K).numpy())
    offsets = np.concatenate([[0], np.sort(r.randint(0, R, E - 1)), [R]]).astype(np.int32)
    dy = torch.from_numpy(r.standard_normal((R, N)).astype(np.float32)).bfloat16()
    w = Q.Mxfp4(torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda"),
                torch.zeros(E, N, K // 32, dtype=torch.uint8, device="cuda"))
    x = Q.Mxfp4(torch.from_numpy(xq[0]).cuda(), torch.from_numpy(xq[1]).cuda())
    off = torch.from_numpy(offsets).cuda()
    _, dw = Q.mxfp4_matmul_backward(dy.cuda(), x, w, off, need_dx=False)
    assert Q.qbmoe_status(None, None) == 0
    some = np.unique(np.concatenate([np.arange(0, N, 37), [N - 1]]))
    for e, (a, b) in enumerate(M.groups(offsets, R)):
        want = dy[a:b].double().numpy()[:, some].T @ xq[2][a:b]
        got = dw[e, some].double().cpu().numpy()
        assert np.linalg.norm(got - want) < 1e-6 * np.linalg.norm(want)
    _, again = Q.mxfp4_matmul_backward(dy.cuda(), x, w, off, need_dx=False)
    assert torch.equal(dw, again)
    _, half = Q.mxfp4_matmul_backward(dy.cuda(), x, w, off, need_dx=False, dw_dtype=torch.bfloat16)
    assert float((half.float() - dw).norm() / dw.norm()) < 2.0 ** -8


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_product_quantises_its_rows(dtype):
    import quantile_balanced_routing_gb300 as Q
    xq, wq, offsets, _ = product_case(611, 24, 264, 544, 2.0)
    _, w, off = on_gpu(Q, xq, wq, offsets, 24, 264, 544)
    x = rows(np.random.RandomState(1), 611, 544).to(getattr(torch, dtype)).cuda()
    y = Q.mxfp4_matmul(x, w, off)
    assert torch.equal(y, Q.mxfp4_matmul(Q.mxfp4_quantize(x), w, off))
    wide = torch.zeros(611, 640, dtype=x.dtype, device="cuda")
    wide[:, 96:] = x
    assert torch.equal(y, Q.mxfp4_matmul(wide[:, 96:], w, off))


def test_gradients_against_differences():
    """Small whole numbers, so that every product, sum and rounding is exact: moving one value of x (or of w) from
    1 to 2 changes sum(dy * y) by exactly that value's gradient."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(0)
    R, N, K = 6, 16, 64
    x = np.where(r.random_sample((R, K)) < 0.2, 1.0, 0.0) * r.choice([-1, 1], (R, K))
    w = r.choice([-2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 2.0], (N, K))
    x[:, ::32] = 4.0                     # every block keeps the scale 2^0
    w[:, ::32] = 4.0
    x[2, 5] = x[5, 40] = w[3, 7] = w[15, 63] = 1.0
    dy = r.choice([-2.0, -1.0, 1.0, 2.0], (R, N))
    t = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731

    def total(x, w):
        return float((t(dy) * Q.mxfp4_matmul(t(x), Q.mxfp4_quantize(t(w))).float()).double().sum())

    base = total(x, w)
    dx, dw = Q.mxfp4_matmul_backward(t(dy).bfloat16(), Q.mxfp4_quantize(t(x)), Q.mxfp4_quantize(t(w)))
    for i, j in ((2, 5), (5, 40)):
        y = x.copy()
        y[i, j] = 2.0
        assert total(y, w) - base == float(dx[i, j])
    for i, j in ((3, 7), (15, 63)):
        y = w.copy()
        y[i, j] = 2.0
        assert total(x, y) - base == float(dw[i, j])


def test_rows_of_other_experts_and_not_finite_values_stay_apart():
    """A row whose codes stand for NaN reaches its own outputs and its expert's weight gradient only."""
    import quantile_balanced_routing_gb300 as Q
    R, E, N, K = 100, 4, 72, 160
    xq, wq, _, dy = product_case(R, E, N, K, 0.0)
    offsets = np.array([0, 37, 37, 70, 100], np.int32)
    x, w, off = on_gpu(Q, xq, wq, offsets, E, N, K)
    clean_y = Q.mxfp4_matmul(x, w, off)
    dx0, dw0 = Q.mxfp4_matmul_backward(dy.cuda(), x, w, off)
    x.scales[37, 2] = 255                  # the first row of expert 2
    dy[69, 5] = float("inf")               # the last row of expert 2
    y = Q.mxfp4_matmul(x, w, off)
    assert torch.isnan(y[37]).all()
    keep = torch.arange(R, device="cuda") != 37
    assert torch.equal(y[keep], clean_y[keep])
    dx, dw = Q.mxfp4_matmul_backward(dy.cuda(), x, w, off)
    keep = torch.arange(R, device="cuda") != 69
    assert torch.equal(dx[keep], dx0[keep])
    for e in (0, 1, 3):
        assert torch.equal(dw[e], dw0[e])
    assert not torch.isfinite(dw[2]).all()
    assert not dw[1].any()


def test_extreme_scales():
    """Blocks near both ends of E8M0 whose products are ordinary numbers."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(2)
    R, N, K = 20, 24, 96
    xq, wq, _, dy = product_case(R, 0, N, K, 0.0)
    xs, ws = xq[1].copy(), wq[1].copy()
    xs[:, 1], ws[:, 1] = 127 + 100, 127 - 101
    xs[:, 2], ws[:, 2] = 13, 127 + 113
    xs[3, 0] = 0                            # 2^-127: no normal fp32 number
    x, w, _ = on_gpu(Q, (xq[0], xs), (wq[0], ws), None, 0, N, K)
    xv, wv = M.decode(xq[0], xs), M.decode(wq[0], ws)
    want, mags = M.matmul(xv, wv[None], None)
    near(Q.mxfp4_matmul(x, w), want, mags, K, True)
    d = dy.double().numpy()
    dx, dw = Q.mxfp4_matmul_backward(dy.cuda(), x, w)
    (wx, mx), (ww, mw) = M.matmul_backward(d, xv, wv[None], None)
    # dx's smallest numbers are below bf16's normal range, where its step is 2^-133
    got = dx.double().cpu().numpy()
    assert (np.abs(got - wx) <= N * 2.0 ** -24 * mx + 2.0 ** -8 * np.abs(wx) + 2.0 ** -133).all()
    got = dw.double().cpu().numpy()
    assert (np.abs(got - ww[0]) <= R * 2.0 ** -24 * mw[0] + 2.0 ** -24 * np.abs(ww[0]) + 2.0 ** -126).all()


def test_no_rows():
    import quantile_balanced_routing_gb300 as Q
    xq, wq, _, _ = product_case(4, 3, 16, 64, 0.0)
    x, w, _ = on_gpu(Q, xq, wq, None, 3, 16, 64)
    none = Q.Mxfp4(x.codes[:0], x.scales[:0])
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert Q.mxfp4_matmul(none, w, off).shape == (0, 16)
    dx, dw = Q.mxfp4_matmul_backward(torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda"), none, w, off)
    assert dx.shape == (0, 64) and dw.shape == (3, 16, 64) and not dw.any()


def test_strided_gradient_rows_repeat_and_other_stream():
    import quantile_balanced_routing_gb300 as Q
    xq, wq, offsets, dy = product_case(611, 24, 264, 544, 2.0)
    x, w, off = on_gpu(Q, xq, wq, offsets, 24, 264, 544)
    wide = torch.full((611, 320), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:272] = dy.cuda()
    a = Q.mxfp4_matmul_backward(dy.cuda(), x, w, off) + (Q.mxfp4_matmul(x, w, off),)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = Q.mxfp4_matmul_backward(wide[:, 8:272], x, w, off, stream=s) + (Q.mxfp4_matmul(x, w, off, stream=s),)
    s.synchronize()
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    only_dx = Q.mxfp4_matmul_backward(dy.cuda(), x, w, off, need_dw=False)
    assert only_dx[1] is None and torch.equal(only_dx[0], a[0])


def test_output_stride_and_rows_without_an_expert():
    """The C entry with a wide y: columns past N, and rows past the last offset, stay as they were."""
    import quantile_balanced_routing_gb300 as Q
    R, E, N, K = 90, 2, 40, 96
    xq, wq, _, _ = product_case(R, E, N, K, 0.0)
    offsets = np.array([0, 33, 80], np.int32)
    x, w, off = on_gpu(Q, xq, wq, offsets, E, N, K)
    lib = Q.load_library()
    y = torch.full((R, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    rc = lib.moe_mxfp4_matmul(R, E, N, K, Q.QBMOE_MXFP4, x.codes.data_ptr(), K,
                              *(t.data_ptr() for t in (x.scales, w.codes, w.scales, off, y)), 64, None, 0, None)
    torch.cuda.synchronize()
    assert rc == 0
    want, mags = M.matmul(xq[2], wq[2].reshape(E, N, K), offsets)
    near(y[:80, :N], want[:80], mags[:80], K, True)
    assert (y[:, N:] == 7).all() and (y[80:] == 7).all()


@pytest.mark.slow
def test_offsets_past_32_bits():
    """Weights and weight gradients of more than 2^32 bytes: the last expert's rows are the ones that matter."""
    import quantile_balanced_routing_gb300 as Q
    E, N, K, R = 400, 1024, 4096, 8           # dw: 6.7 GB
    g = torch.Generator(device="cuda").manual_seed(0)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(118, 124, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    w = Q.Mxfp4(codes, scales)
    r = np.random.RandomState(0)
    xq = M.quantize(rows(r, R, K).numpy())
    x = Q.Mxfp4(torch.from_numpy(xq[0]).cuda(), torch.from_numpy(xq[1]).cuda())
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E:] = R
    y = Q.mxfp4_matmul(x, w, off)
    wv = M.decode(codes[-1].cpu().numpy(), scales[-1].cpu().numpy())
    want, mags = M.matmul(xq[2], wv[None], None)
    near(y, want, mags, K, True)
    dy = torch.from_numpy(r.standard_normal((R, N)).astype(np.float32)).bfloat16()
    dx, dw = Q.mxfp4_matmul_backward(dy.cuda(), x, w, off)
    (wx, mx), (ww, mw) = M.matmul_backward(dy.double().numpy(), xq[2], wv[None], None)
    near(dx, wx, mx, N, True)
    near(dw[-1], ww[0], mw[0], R, False)
    assert not dw[:-1].any()


def test_bounded_wait_reports_and_recovers():
    """The issuer withholds its first accumulator: the waits run out, the status says so, the next call is right."""
    import quantile_balanced_routing_gb300 as Q
    lib = Q.load_library()
    xq, wq, offsets, dy = product_case(611, 24, 264, 544, 2.0)
    x, w, off = on_gpu(Q, xq, wq, offsets, 24, 264, 544)
    dy = dy.cuda()
    calls = [lambda: Q.mxfp4_matmul(x, w, off), lambda: Q.mxfp4_matmul_backward(dy, x, w, off, need_dw=False)[0],
             lambda: Q.mxfp4_matmul_backward(dy, x, w, off, need_dx=False)[1]]
    want = [f() for f in calls]
    assert Q.qbmoe_status(None, None) == 0
    for f, right in zip(calls, want):
        lib.qbmoe_set_wait_limit(None, 200)
        lib.qbmoe_debug_stall(None, 1)
        try:
            f()
            assert Q.qbmoe_status(None, None) == Q.QBMOE_ETIMEOUT
        finally:
            lib.qbmoe_debug_stall(None, 0)
            lib.qbmoe_set_wait_limit(None, 0)
        assert Q.qbmoe_status(None, None) == 0
        assert torch.equal(f(), right)
        assert Q.qbmoe_status(None, None) == 0


@pytest.mark.parametrize("K", [512, 544, 96])
def test_gradients_decode_every_code_and_scale(K):
    """With the identity as dy the gradients are the operands' values, exactly, at every scale whose
    values are normal and finite (blocks of a row take scales 37 apart)."""
    import quantile_balanced_routing_gb300 as Q
    n = 256
    row, block = np.arange(n)[:, None], np.arange(K // 32)[None]
    scales = (2 + (row + 37 * block) % 251).astype(np.uint8)          # 2 .. 252
    byte = (np.arange(K // 2)[None] * 17 + 5 * row) % 256               # both codes of a byte, all pairs
    codes = byte.astype(np.uint8)
    q, _, _ = on_gpu(Q, (codes, scales), (codes, scales), None, 0, n, K)
    want = M.decode(codes, scales)
    dx, dw = Q.mxfp4_matmul_backward(torch.eye(n).bfloat16().cuda(), q, q)
    assert np.array_equal(dx.double().cpu().numpy(), want)
    assert np.array_equal(dw.double().cpu().numpy(), want)


@pytest.mark.parametrize("R,N,K", [(208, 152 * 128, 96), (203, 152 * 128 - 56, 512), (386, 76 * 128, 544)])
def test_product_of_one_matrix_in_fewer_rounds(R, N, K):
    """Rows that tiles of 208 hold in one round of the grid less than tiles of 192."""
    import quantile_balanced_routing_gb300 as Q
    xq, wq, _, _ = product_case(R, 0, N, K, 0.0)
    x, w, _ = on_gpu(Q, xq, wq, None, 0, N, K)
    want, mags = M.matmul(xq[2], wq[2][None], None)
    near(Q.mxfp4_matmul(x, w), want, mags, K, True)
    assert Q.qbmoe_status(None, None) == 0
