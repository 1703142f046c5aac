"""moe_mxfp4_matvec and moe_mxfp4_experts against their definitions in 64 bits.

Products of E2M1 codes with bf16 or E4M3 elements are exact in fp32, so a product differs from
the exact sum by its fp32 additions, at most K 2^-24 of the sum of magnitudes, by what the blocks'
fp16 form drops (2^-40 of a block's largest) and by the rounding of the output.
"""
import numpy as np
import pytest

import few_rows_reference as F
import mx_reference as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return t.double().cpu().numpy()


def near(got, want, bound):
    got = f64(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


def rows(r, R, K, kind):
    """(what the call takes, 64-bit values): rows with a scale of their own, a block of zeros, tiny elements."""
    import quantile_balanced_routing_gb300 as Q
    x = r.standard_normal((R, K)) * np.exp(r.standard_normal((R, 1)))
    x[:, ::7] *= 1e-5
    if R:
        x[R // 2, :32] = 0.0
    if kind == "bf16":
        t = torch.from_numpy(x).to(torch.bfloat16)
        return t.cuda(), f64(t)
    codes, scales = F.quantize8(x)
    return Q.Mxfp8(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()), F.decode8(codes, scales)


def cuda(*arrays):
    return [torch.from_numpy(a).cuda() for a in arrays]


def weights(r, *shape):
    import quantile_balanced_routing_gb300 as Q
    c, s, v = F.weights(r, *shape)
    return Q.Mxfp4(*cuda(c, s)), v


def grouped(x, w, offsets):
    y, b = np.zeros((x.shape[0], w.shape[1])), np.zeros((x.shape[0], w.shape[1]))
    for e, (lo, hi) in enumerate(M.groups(offsets, x.shape[0])):
        if hi > lo:
            y[lo:hi], b[lo:hi] = F.product(x[lo:hi], w[e])
    return y, b


@pytest.mark.parametrize("kind", ["bf16", "mxfp8"])
@pytest.mark.parametrize("R,N,K", [(1, 8, 32), (1, 264, 544), (3, 24, 96), (7, 40, 1024), (8, 136, 480), (9, 72, 2048),
                                   (17, 16, 512), (33, 48, 1056), (1, 1024, 7168), (13, 896, 3584), (2, 8, 8192),
                                   (5, 24, 8224), (1, 16, 20000 // 32 * 32), (12, 32, 4128), (16, 8, 65536)])
def test_dense(R, N, K, kind):
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(R + N + K)
    x, xv = rows(r, R, K, kind)
    w, wv = weights(r, N, K)
    want, bound = F.product(xv, wv)
    for dtype in (torch.float32, torch.bfloat16):
        y = Q.mxfp4_matvec(x, w, out_dtype=dtype)
        assert y.dtype == dtype
        near(y, want, bound + HALF[dtype] * np.abs(want))
    assert torch.equal(Q.mxfp4_matvec(x, w), y)


@pytest.mark.parametrize("kind", ["bf16", "mxfp8"])
@pytest.mark.parametrize("loads,N,K", [([3], 8, 32), ([0, 5, 0, 0, 1], 24, 96), ([1] * 40, 16, 64), ([0, 0], 8, 64),
                                       ([61, 0, 7, 8, 9, 16, 17], 264, 544), ([2, 0, 130], 40, 1056),
                                       ([5] * 100 + [0] * 20 + [11], 64, 3584), ([1, 2, 3], 1000, 8320)])
def test_grouped(loads, N, K, kind):
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(len(loads) + N + K)
    off = np.concatenate([[0], np.cumsum(loads)]).astype(np.int32)
    x, xv = rows(r, int(off[-1]), K, kind)
    w, wv = weights(r, len(loads), N, K)
    want, bound = grouped(xv, wv, off)
    y = Q.mxfp4_matvec(x, w, offsets=cuda(off)[0], out_dtype=torch.float32)
    near(y, want, bound + HALF[torch.float32] * np.abs(want))
    y = Q.mxfp4_matvec(x, w, offsets=cuda(off)[0])
    near(y, want, bound + HALF[torch.bfloat16] * np.abs(want))


def call(x, K, w, offsets, y, ldx=None):
    """The C entry with the caller's own output."""
    import quantile_balanced_routing_gb300 as Q
    E, N = (w.shape[0], w.shape[1]) if offsets is not None else (1, w.shape[0])
    lib = Q.load_library()
    need = lib.qbmoe_mxfp4_matvec_workspace_bytes(x.shape[0], N, K)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    return lib.moe_mxfp4_matvec(x.shape[0], E, N, K, 1, x.data_ptr(), ldx or x.stride(0), None, w.codes.data_ptr(),
                                w.scales.data_ptr(), None if offsets is None else offsets.data_ptr(),
                                0 if y.dtype == torch.float32 else 1, y.data_ptr(), y.stride(0), ws.data_ptr(), need,
                                torch.cuda.current_stream().cuda_stream or None)


@pytest.mark.parametrize("K", [96, 8256])
def test_rows_without_an_expert_and_the_space_between_rows_stay(K):
    r = np.random.RandomState(K)
    w, wv = weights(r, 3, 24, K)
    t = torch.from_numpy(r.standard_normal((20, K + 24))).to(torch.bfloat16).cuda()
    x = t[:, 8:8 + K]
    for off in ([4, 4, 9, 15], [0, 3, 3, 3], [20, 20, 20, 20]):
        y = torch.full((20, 33), 7.0, device="cuda")
        assert call(x, K, w, cuda(np.array(off, np.int32))[0], y) == 0
        lo, hi = off[0], off[-1]
        want, bound = grouped(f64(x)[lo:hi], wv, np.array(off) - lo)
        near(y[lo:hi, :24], want, bound + 2.0 ** -24 * np.abs(want))
        assert (y[:lo] == 7).all() and (y[hi:] == 7).all() and (y[:, 24:] == 7).all()


def test_every_code_scale_and_a_scale_of_nan():
    """Weights of single nonzero blocks, so that a product is one code times one scale."""
    import quantile_balanced_routing_gb300 as Q
    K, N = 64, 256 * 8
    codes = np.zeros((N, K // 2), np.uint8)
    scales = np.full((N, 2), 127, np.uint8)
    scales[:, 0] = np.repeat(np.arange(256), 8)
    codes[:, 3] = np.tile(np.arange(8) * 2 + 1, 256) | (np.tile(np.arange(8) * 2, 256) << 4)
    x = np.zeros((2, K))
    x[0, 6], x[1, 7] = 1.0, -2.0
    y = Q.mxfp4_matvec(torch.from_numpy(x).to(torch.bfloat16).cuda(), Q.Mxfp4(*cuda(codes, scales)), out_dtype=torch.float32)
    want = x @ M.decode(codes, scales).T
    got = f64(y)
    nan = np.repeat(np.arange(256) == 255, 8)
    assert np.isnan(got[:, nan]).all()
    fine = ~nan & (np.abs(want) < 3.4e38).all(0)
    assert np.array_equal(got[:, fine], want[:, fine])
    assert (np.isinf(got) == (np.abs(want) > 3.4e38))[:, ~nan].all()


def test_rows_of_large_small_and_bad_elements():
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(0)
    w, wv = weights(r, 40, 128)
    x = r.standard_normal((9, 128))
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2, :32] *= 1e20
    x[3, 5] = 1e9                     # a block whose other elements are 2^-30 of its largest
    x[4], x[5, 40] = 0.0, np.inf
    x[6, 41], x[7, 50], x[7, 51] = np.nan, np.inf, -np.inf
    t = torch.from_numpy(x).to(torch.bfloat16)
    y = f64(Q.mxfp4_matvec(t.cuda(), w, out_dtype=torch.float32))
    for i in (0, 1, 2, 3, 4, 8):
        want, bound = F.product(f64(t[i:i + 1]), wv)
        near(torch.from_numpy(y[i:i + 1]), want, bound + 2.0 ** -24 * np.abs(want))
    assert np.isnan(y[6]).all()
    nz = wv[:, 40] != 0
    assert np.array_equal(y[5][nz], np.sign(wv[nz, 40]) * np.inf) and np.isnan(y[5][~nz]).all()
    assert not np.isfinite(y[7]).any()


def test_mxfp8_extremes():
    """Every E4M3 code, and the scales that fp32 holds."""
    import quantile_balanced_routing_gb300 as Q
    codes = np.zeros((256, 32), np.uint8)
    codes[:, 9] = np.arange(256)
    scales = np.full((256, 1), 127, np.uint8)
    c, s, v = M.quantize(np.where(np.arange(32) == 9, 3.0, 1.0)[None].repeat(8, 0))
    y = f64(Q.mxfp4_matvec(Q.Mxfp8(*cuda(codes, scales)), Q.Mxfp4(*cuda(c, s)), out_dtype=torch.float32))
    want = F.decode8(codes, scales) @ v.T
    assert np.array_equal(np.isnan(y), np.isnan(want)) and np.isnan(y).sum() == 16
    assert np.array_equal(np.nan_to_num(y), np.nan_to_num(want))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    codes[:, 9] = 56                  # 1.0
    y = f64(Q.mxfp4_matvec(Q.Mxfp8(*cuda(codes, scales)), Q.Mxfp4(*cuda(c, s)), out_dtype=torch.float32))
    want = 3.0 * np.ldexp(1.0, np.arange(256) - 127)
    fine = (np.arange(256) >= 1) & (np.arange(256) <= 252)
    assert np.array_equal(y[fine], np.repeat(want[fine, None], 8, 1)) and np.isnan(y[255]).all()


def routed(r, T, k, E, distinct=True):
    idx = np.stack([r.permutation(E)[:k] for _ in range(T)]) if distinct else r.randint(0, E, (T, k))
    w = r.random_sample((T, k)) + 0.05
    return idx.astype(np.int32), (w / w.sum(1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("kind", ["bf16", "mxfp8"])
@pytest.mark.parametrize("T,k,E,L,Mi,gamma", [(1, 1, 1, 32, 32, True), (1, 16, 40, 512, 256, True), (3, 2, 5, 96, 160, False),
                                              (7, 4, 33, 544, 96, True), (9, 32, 64, 64, 64, True), (40, 3, 4, 128, 96, False),
                                              (30, 8, 12, 1056, 32, True), (2, 2, 3, 3584, 1024, True), (1, 1, 2, 8256, 64, True),
                                              (3, 2, 4, 64, 8224, True), (128, 32, 200, 32, 32, True)])
def test_experts(T, k, E, L, Mi, gamma, kind):
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(T + k + E + L)
    x, xv = rows(r, T, L, kind)
    (g, gv), (u, uv), (o, ov) = weights(r, E, Mi, L), weights(r, E, Mi, L), weights(r, E, L, Mi)
    idx, w = routed(r, T, k, E)
    gain = (1 + 0.3 * r.standard_normal(L)).astype(np.float32) if gamma else None
    y = Q.mxfp4_experts(x, *cuda(idx, w), g, u, o, gamma=cuda(gain)[0] if gamma else None)
    assert y.dtype == torch.bfloat16
    want, bound = F.experts(xv, idx, w.astype(np.float64), gv, uv, ov, gain, 1e-6)
    near(y, want, bound + 2.0 ** -8 * np.abs(want))
    assert torch.equal(Q.mxfp4_experts(x, *cuda(idx, w), g, u, o, gamma=cuda(gain)[0] if gamma else None), y)


def test_experts_the_same_one_twice_none_and_outside():
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(5)
    E, L, Mi = 6, 64, 96
    x, xv = rows(r, 12, L, "bf16")
    (g, gv), (u, uv), (o, ov) = weights(r, E, Mi, L), weights(r, E, Mi, L), weights(r, E, L, Mi)
    idx, w = routed(r, 12, 4, E, distinct=False)
    idx[0] = 3                                   # one expert four times
    idx[1, 2], idx[2], idx[3, 0] = -1, E, 1 << 30   # no route: one, all, one
    y = Q.mxfp4_experts(x, *cuda(idx, w), g, u, o)
    want, bound = F.experts(xv, idx, w.astype(np.float64), gv, uv, ov, None, 1e-6)
    near(y, want, bound + 2.0 ** -8 * np.abs(want))
    assert not y[2].any()
    y = Q.mxfp4_experts(x, *cuda(idx, w), g, u, o, gamma=torch.ones(L, device="cuda"))
    assert not y[2].any()


def test_experts_other_betas_strides_and_offsets_of_slices():
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(6)
    E, L, Mi = 4, 96, 64
    t = torch.from_numpy(r.standard_normal((5, 128)) * 3).to(torch.bfloat16).cuda()
    x = t[:, 16:16 + L]
    (g, gv), (u, uv), (o, ov) = weights(r, E + 1, Mi, L), weights(r, E + 1, Mi, L), weights(r, E + 1, L, Mi)
    cut = lambda q: Q.Mxfp4(q.codes[1:], q.scales[1:])  # noqa: E731
    idx, w = routed(r, 5, 3, E)
    y = Q.mxfp4_experts(x, *cuda(idx, w), cut(g), cut(u), cut(o), beta1=1.5, beta2=3.0)
    want, bound = F.experts(f64(x), idx, w.astype(np.float64), gv[1:], uv[1:], ov[1:], None, 1e-6, 1.5, 3.0)
    near(y, want, bound + 2.0 ** -8 * np.abs(want))


def test_a_bad_token_stays_in_its_row():
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(7)
    (g, _), (u, _), (o, _) = weights(r, 3, 64, 64), weights(r, 3, 64, 64), weights(r, 3, 64, 64)
    x, _ = rows(r, 20, 64, "bf16")
    idx, w = routed(r, 20, 2, 3)
    a = Q.mxfp4_experts(x, *cuda(idx, w), g, u, o)
    x = x.clone()
    x[4, 3], x[9, 60] = float("nan"), float("inf")
    b = Q.mxfp4_experts(x, *cuda(idx, w), g, u, o)
    ok = torch.ones(20, dtype=torch.bool)
    ok[[4, 9]] = False
    assert torch.equal(a[ok.cuda()], b[ok.cuda()]) and torch.isnan(b[4]).all()


def test_no_rows():
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(8)
    (g, _), (u, _), (o, _) = weights(r, 3, 64, 32), weights(r, 3, 64, 32), weights(r, 3, 32, 64)
    x = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    i, w = torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda")
    assert Q.mxfp4_experts(x, i, w, g, u, o).shape == (0, 32)
    assert Q.mxfp4_matvec(x, Q.Mxfp4(g.codes[0], g.scales[0])).shape == (0, 64)
    assert Q.mxfp4_matvec(x, g, offsets=torch.zeros(4, dtype=torch.int32, device="cuda")).shape == (0, 64)


@pytest.mark.parametrize("K", [256, 8448])
def test_captured_replayed_and_on_two_streams(K):
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(9)
    E, Mi = 8, 128
    (g, _), (u, _), (o, _) = weights(r, E, Mi, K), weights(r, E, Mi, K), weights(r, E, K, Mi)
    x, _ = rows(r, 6, K, "bf16")
    idx, w = cuda(*routed(r, 6, 3, E))
    off = cuda(np.array([0, 1, 1, 2, 3, 3, 4, 6, 6], np.int32))[0]
    run = lambda s=None: (Q.mxfp4_matvec(x, g, offsets=off, stream=s), Q.mxfp4_experts(x, idx, w, g, u, o, stream=s))  # noqa: E731
    want = run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [run(s) for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for pair in got for a, b in zip(pair, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    x.copy_(rows(r, 6, K, "bf16")[0])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, run()))


def test_a_decode_step_of_a_block():
    """Residual and norm in 8 bits, router logits, routing, latent rows, experts, up-projection: as a layer runs them."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(10)
    T, d, L, Mi, E, k = 5, 256, 128, 96, 24, 4
    gain = (1 + 0.2 * r.standard_normal(d)).astype(np.float32)
    lat = (1 + 0.2 * r.standard_normal(L)).astype(np.float32)
    (wr, wrv), (wd, wdv), (wu, wuv) = weights(r, E, d), weights(r, L, d), weights(r, d, L)
    (g, gv), (u, uv), (o, ov) = weights(r, E, Mi, L), weights(r, E, Mi, L), weights(r, E, L, Mi)
    x, stream = (torch.from_numpy(r.standard_normal((T, d))).to(torch.bfloat16).cuda() for _ in range(2))
    n = Q.add_rmsnorm(x, cuda(gain)[0], residual=stream, mxfp8=True, total=stream)
    logits = Q.mxfp4_matvec(n.q, wr, out_dtype=torch.float32)
    h = Q.mxfp4_matvec(n.q, wd)
    _, _, idx, w, _ = Q.route_qb(logits, k, qb_sweeps=0)
    z = Q.mxfp4_experts(h, idx, w, g, u, o, gamma=cuda(lat)[0])
    y = Q.mxfp4_matvec(z, wu)
    # each step against its definition on what the step before it gave
    nv = F.decode8(n.q.codes.view(torch.uint8).cpu().numpy(), n.q.scales.cpu().numpy())
    assert np.abs(nv - F.norm(f64(stream), gain, 1e-6)).max() <= 2.0 ** -4 * np.abs(nv).max()
    for got, a, b, half in ((logits, nv, wrv, 2.0 ** -24), (h, nv, wdv, 2.0 ** -8), (y, f64(z), wuv, 2.0 ** -8)):
        want, bound = F.product(a, b)
        near(got, want, bound + half * np.abs(want))
    s = 1 / (1 + np.exp(-f64(logits)))
    assert np.array_equal(idx.cpu().numpy(), np.argsort(-s, axis=1, kind="stable")[:, :k])
    want, bound = F.experts(f64(h), idx.cpu().numpy(), f64(w), gv, uv, ov, lat, 1e-6)
    near(z, want, bound + 2.0 ** -8 * np.abs(want))
    assert Q.qbmoe_status(None, None) == 0


@pytest.mark.parametrize("N,K", [(65536, 64), (32768, 256), (32768, 512), (24576, 1024), (16384, 2048), (8192, 3584), (8192, 4096), (4096, 7168)])
def test_many_tiles(N, K):
    """Each stage of the weights' ring is filled many times, also with groups of warps at different paces."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(N)
    off = np.array([0, 3, 3, 5, 14], np.int32)
    x, xv = rows(r, 14, K, "mxfp8")
    codes = torch.randint(0, 256, (4, N, K // 2), dtype=torch.uint8, device="cuda", generator=torch.Generator("cuda").manual_seed(N))
    scales = torch.randint(110, 124, (4, N, K // 32), dtype=torch.uint8, device="cuda", generator=torch.Generator("cuda").manual_seed(K))
    w = Q.Mxfp4(codes, scales)
    first = Q.mxfp4_matvec(x, w, offsets=cuda(off)[0], out_dtype=torch.float32)
    for _ in range(20):
        assert torch.equal(Q.mxfp4_matvec(x, w, offsets=cuda(off)[0], out_dtype=torch.float32), first)
    some = r.choice(N, 300, replace=False)
    wv = M.decode(codes.cpu().numpy()[:, some], scales.cpu().numpy()[:, some])
    want, bound = grouped(xv, wv, off)
    near(first[:, torch.from_numpy(some).cuda()], want, bound + HALF[torch.float32] * np.abs(want))


# Calls whose rows become sums of MXFP4 rows: from 2^26 elements of weights on, read once and per eight rows again.
# A bf16 element is then within 2^-22 of its block's largest: 2^-22 sum_b max_b sum_(k in b) |w| more.
def in_pieces(n, R, N, K):
    return (n + R // 8) * N * K >= 1 << 26


# (In the experts' bound that is far inside the additions' term, K 2^-24 of the sum of magnitudes, as K >= 512; the
# SiTU-GLU's result keeps 2^-22 where the bound allows 2^-12.)
def dropped(xv, wv):
    """2^-22 of each block's largest, times the block's weights."""
    R, K = xv.shape
    return 2.0 ** -22 * np.abs(xv).reshape(R, K // 32, 32).max(2) @ np.abs(wv).reshape(-1, K // 32, 32).sum(2).T


@pytest.mark.parametrize("kind", ["bf16", "mxfp8"])
@pytest.mark.parametrize("R,N,K", [(1000, 648, 1024), (2101, 648, 768), (4100, 640, 256), (67, 1048, 7168), (700, 264, 8192)])
def test_dense_in_pieces(R, N, K, kind):
    import quantile_balanced_routing_gb300 as Q
    assert in_pieces(1, R, N, K)
    r = np.random.RandomState(R + N + K)
    x, xv = rows(r, R, K, kind)
    w, wv = weights(r, N, K)
    want, bound = F.product(xv, wv)
    bound = bound + dropped(xv, wv)
    for dtype in (torch.float32, torch.bfloat16):
        y = Q.mxfp4_matvec(x, w, out_dtype=dtype)
        near(y, want, bound + HALF[dtype] * np.abs(want))
    assert torch.equal(Q.mxfp4_matvec(x, w), y)


@pytest.mark.parametrize("kind", ["bf16", "mxfp8"])
@pytest.mark.parametrize("loads,N,K", [([1, 0, 2, 3] * 100, 144, 1024), ([0, 5, 9, 0, 1, 30, 7, 8] * 20, 328, 768),
                                       ([40, 0, 1, 100, 3] * 12, 264, 1280), ([300, 0, 25, 513], 648, 1024)])
def test_grouped_in_pieces(loads, N, K, kind):
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(len(loads) + N + K)
    off = np.concatenate([[0], np.cumsum(loads)]).astype(np.int32)
    assert in_pieces(min(len(loads), off[-1]), off[-1], N, K)
    x, xv = rows(r, int(off[-1]), K, kind)
    w, wv = weights(r, len(loads), N, K)
    want, bound = grouped(xv, wv, off)
    for e, (lo, hi) in enumerate(M.groups(off, off[-1])):
        if hi > lo:
            bound[lo:hi] += dropped(xv[lo:hi], wv[e])
    for dtype in (torch.float32, torch.bfloat16):
        near(Q.mxfp4_matvec(x, w, offsets=cuda(off)[0], out_dtype=dtype), want, bound + HALF[dtype] * np.abs(want))


def test_rows_without_an_expert_and_the_space_between_rows_stay_in_pieces():
    r = np.random.RandomState(1)
    R, N, K = 1100, 648, 768
    assert in_pieces(3, R, N, K)
    w, wv = weights(r, 3, N, K)
    t = torch.from_numpy(r.standard_normal((R, K + 24))).to(torch.bfloat16).cuda()
    x = t[:, 8:8 + K]
    for off in ([4, 4, 9, 1015], [0, 903, 903, 903], [R, R, R, R]):
        x[:off[0]], x[off[3]:] = float("nan"), float("inf")   # nobody's
        y = torch.full((R, N + 9), 7.0, device="cuda")
        assert call(x, K, w, cuda(np.array(off, np.int32))[0], y) == 0
        lo, hi = off[0], off[-1]
        want, bound = grouped(f64(x)[lo:hi], wv, np.array(off) - lo)
        if hi > lo:
            bound += np.maximum.reduce([dropped(f64(x)[lo:hi], wv[e]) for e in range(3)])
        near(y[lo:hi, :N], want, bound + 2.0 ** -24 * np.abs(want))
        assert (y[:lo] == 7).all() and (y[hi:] == 7).all() and (y[:, N:] == 7).all()
        t.copy_(torch.from_numpy(r.standard_normal((R, K + 24))).to(torch.bfloat16))
    y = torch.zeros(R, N, device="cuda")   # offsets out of order and out of range stay in their tensors
    assert call(x, K, w, cuda(np.array([-5, 1 << 30, 7, R + 9], np.int32))[0], y) == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("infinite", [False, True])
def test_bad_rows_in_pieces(infinite):
    """Rows with infinities or tiny blocks have no pieces and are multiplied as they are; no row touches another."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(2)
    R, N, K = 1000, 648, 1024
    w, wv = weights(r, N, K)
    x = r.standard_normal((R, K))
    x[0] *= 1e30
    x[1] *= 1e-20
    x[2, :32] *= 1e20
    x[4], x[6, 41] = 0.0, np.nan
    before = Q.mxfp4_matvec(torch.from_numpy(x).to(torch.bfloat16).cuda(), w, out_dtype=torch.float32)
    if infinite:
        x[1] *= 1e-12
        x[5, 40], x[7, 50], x[7, 51] = np.inf, np.inf, -np.inf
    t = torch.from_numpy(x).to(torch.bfloat16)
    y = f64(Q.mxfp4_matvec(t.cuda(), w, out_dtype=torch.float32))
    fine = [i for i in range(R) if i not in ((5, 6, 7) if infinite else (6,))]
    want, bound = F.product(f64(t)[fine], wv)
    near(torch.from_numpy(y[fine]), want, bound + dropped(f64(t)[fine], wv) + 2.0 ** -24 * np.abs(want))
    assert np.isnan(y[6]).all()
    if infinite:
        nz = wv[:, 40] != 0
        assert np.array_equal(y[5][nz], np.sign(wv[nz, 40]) * np.inf) and np.isnan(y[5][~nz]).all()
        assert not np.isfinite(y[7]).any()
    same = [i for i in range(R) if i not in (1, 5, 6, 7)]
    assert np.array_equal(y[same], f64(before)[same])


def test_mxfp8_extremes_in_pieces():
    """Every E4M3 code but the NaNs, alone in its block, and scales in range and out of it."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(3)
    R, N, K = 2048, 640, 512
    codes = np.zeros((R, K), np.uint8)
    codes[np.arange(R), r.randint(0, K, R)] = np.arange(R) % 256
    codes[codes & 127 == 127] = 1
    w, wv = weights(r, N, K)
    for lo, hi in ((118, 136), (20, 230), (0, 254)):
        scales = r.randint(lo, hi + 1, (R, K // 32)).astype(np.uint8)
        xv = F.decode8(codes, scales)
        y = f64(Q.mxfp4_matvec(Q.Mxfp8(*cuda(codes, scales)), w, out_dtype=torch.float32))
        want = xv @ wv.T
        # an element times a code of up to 6, before the weight's scale (2^-7 to 2^-5), is an fp32 number:
        # beyond 2^128 it is infinite, though the product would be finite
        fine = (np.abs(want) < 1e38) & ((np.abs(want) > 1e-36) | (want == 0)) & (6 * np.abs(xv).max(1) < 2.0 ** 128)[:, None]
        assert np.array_equal(y[fine], want[fine].astype(np.float32))
    scales[9, 3] = 255
    y = Q.mxfp4_matvec(Q.Mxfp8(*cuda(codes, scales)), w)
    assert torch.isnan(y[9]).all() and not torch.isnan(y[10:]).any()


@pytest.mark.parametrize("kind", ["bf16", "mxfp8"])
@pytest.mark.parametrize("T,k,E,L,Mi,gamma", [(100, 8, 16, 768, 512, True), (1, 16, 40, 2048, 768, False), (260, 4, 7, 512, 512, True),
                                              (33, 32, 40, 1024, 256, True)])
def test_experts_in_pieces(T, k, E, L, Mi, gamma, kind):
    import quantile_balanced_routing_gb300 as Q
    assert in_pieces(min(E, T * k), T * k, 3 * L, Mi)
    r = np.random.RandomState(T + k + E + L)
    x, xv = rows(r, T, L, kind)
    (g, gv), (u, uv), (o, ov) = weights(r, E, Mi, L), weights(r, E, Mi, L), weights(r, E, L, Mi)
    idx, w = routed(r, T, k, E, distinct=k <= E)
    if T > 9:
        idx[0] = 3                                                  # one expert k times
        idx[1, 2], idx[2], idx[3, 0] = -1, E, 1 << 30               # no route: one, all, one
    gain = (1 + 0.3 * r.standard_normal(L)).astype(np.float32) if gamma else None
    run = lambda: Q.mxfp4_experts(x, *cuda(idx, w), g, u, o, gamma=cuda(gain)[0] if gamma else None)  # noqa: E731
    y = run()
    want, bound = F.experts(xv, idx, w.astype(np.float64), gv, uv, ov, gain, 1e-6)
    near(y, want, bound + 2.0 ** -8 * np.abs(want))
    assert torch.equal(run(), y) and (T <= 9 or not y[2].any())
    if kind == "bf16" and T > 9:   # a token with an infinity, and one with a NaN
        x = x.clone()
        x[4, 3], x[5, 60] = float("inf"), float("nan")
        bad = run()
        keep = [t for t in range(T) if t not in (4, 5)]
        assert torch.equal(bad[keep], y[keep]) and torch.isnan(bad[5]).all()


def test_in_pieces_captured_replayed_and_on_two_streams():
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(4)
    E, L, Mi, T, k = 16, 768, 512, 100, 8
    (g, _), (u, _), (o, _) = weights(r, E, Mi, L), weights(r, E, Mi, L), weights(r, E, L, Mi)
    x, _ = rows(r, T, L, "bf16")
    many, _ = rows(r, 1400, L, "bf16")
    idx, w = cuda(*routed(r, T, k, E))
    off = torch.linspace(0, 1400, E + 1, device="cuda").to(torch.int32)
    assert in_pieces(E, 1400, Mi, L) and in_pieces(E, T * k, 3 * L, Mi)
    run = lambda s=None: (Q.mxfp4_matvec(many, g, offsets=off, stream=s), Q.mxfp4_experts(x, idx, w, g, u, o, stream=s))  # noqa: E731
    want = run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [run(s) for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for pair in got for a, b in zip(pair, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    x.copy_(rows(r, T, L, "bf16")[0])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, run()))
    x[3, 3] = float("inf")           # the replayed graph decides anew
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) for a, b in zip(captured, run()))
    assert Q.qbmoe_status(None, None) == 0


def test_routing_of_logits_in_pieces():
    """Kernels that are launched while the one before them drains see all of the products."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(11)
    T, n, K = 1500, 896, 1024
    assert in_pieces(1, T, n, K)
    w, _ = weights(r, n, K)
    batches = [torch.from_numpy(r.standard_normal((T, K))).to(torch.bfloat16).cuda() for _ in range(4)]
    want = []
    for x in batches:
        logits = Q.mxfp4_matvec(x, w, out_dtype=torch.float32)
        torch.cuda.synchronize()
        want.append([t.clone() for t in Q.route_qb(logits, 16)])
        torch.cuda.synchronize()
    for _ in range(10):
        for x, expect in zip(batches, want):
            got = Q.route_qb(Q.mxfp4_matvec(x, w, out_dtype=torch.float32), 16)
            assert all(torch.equal(a, b) for a, b in zip(got, expect))


@pytest.mark.parametrize("R", [131072, 131080])
def test_most_rows_in_pieces_and_beyond(R):
    """2^25 elements of x are split; more are multiplied as they are."""
    import quantile_balanced_routing_gb300 as Q
    N, K = 32, 256
    assert in_pieces(1, R, N, K)
    r = np.random.RandomState(12)
    w, wv = weights(r, N, K)
    x = torch.randn(R, K, device="cuda", generator=torch.Generator("cuda").manual_seed(R)).to(torch.bfloat16)
    y = Q.mxfp4_matvec(x, w, out_dtype=torch.float32).double()
    wt = torch.from_numpy(wv).cuda()
    want = x.double() @ wt.T
    top = x.double().abs().view(R, K // 32, 32).amax(2)
    bound = (K + 1) * 2.0 ** -24 * (x.double().abs() @ wt.abs().T) + 2.0 ** -22 * (top @ wt.abs().view(N, K // 32, 32).sum(2).T)
    assert ((y - want).abs() <= bound).all()


def test_no_row_has_pieces():
    """The slow way for every row of the deepest product ends in time for the kernel's waits."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(13)
    R, N, K = 700, 264, 8192
    assert in_pieces(1, R, N, K)
    w, wv = weights(r, N, K)
    x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    x[:, ::32] = 2.0 ** -110                     # below what the scales follow
    y = Q.mxfp4_matvec(x, w, out_dtype=torch.float32)
    want = 2.0 ** -110 * wv[:, ::32].sum(1)
    near(y, np.repeat(want[None], R, 0), K * 2.0 ** -24 * 2.0 ** -110 * np.abs(wv[:, ::32]).sum(1)[None].repeat(R, 0))
    assert Q.qbmoe_status(None, None) == 0
