"""Few-row products and experts on inputs whose results single out one element, digit, route or feature.

Weights of one nonzero code a row make a product one element of x times a power of two, which
fp32 holds: bits can be compared, and nothing hides behind the rounding of a long sum.
"""
import numpy as np
import pytest

import few_rows_reference as F

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def cuda(*arrays):
    return [torch.from_numpy(a).cuda() for a in arrays]


def picks(cols, K, sign=None):
    """(codes, scales) of weights [..., N, K] whose row f is 1 (or sign[f]) at cols[..., f], else 0."""
    c = np.zeros((*cols.shape, K // 2), np.uint8)
    code = 2 + 8 * (np.zeros(cols.shape, np.uint8) if sign is None else (sign < 0).astype(np.uint8))
    np.put_along_axis(c, (cols // 2)[..., None], (code << (4 * (cols % 2))).astype(np.uint8)[..., None], -1)
    return c, np.full((*cols.shape, K // 32), 127, np.uint8)


@pytest.mark.parametrize("E,N,K", [(1, 8, 8224), (1, 520, 8224), (3, 1000, 8224), (5, 264, 8288), (1, 40, 65504)])
def test_the_last_scales_of_deep_rows(E, N, K):
    """Slabs of rows whose scales end off 16 bytes: the tensor's last bytes go one by one."""
    import quantile_balanced_routing_gb300 as Q
    blocks = K // 32
    assert E * N * blocks % 16 == 8
    r = np.random.RandomState(N)
    back = (E * N - 1 - np.arange(E * N)).reshape(E, N) % 8    # row f's only element lies in one of the last eight blocks
    c, s = picks((blocks - 1 - back) * 32 + 5, K)
    s[...] = r.randint(100, 150, s.shape)
    x = np.zeros((E, K))
    x[:, 5::32] = 1.0
    off = cuda(np.arange(E + 1, dtype=np.int32))[0]
    want = np.ldexp(1.0, np.take_along_axis(s, (blocks - 1 - back)[..., None], -1)[..., 0].astype(int) - 127)
    xt, w = torch.from_numpy(x).to(torch.bfloat16).cuda(), Q.Mxfp4(*cuda(c, s))
    for _ in range(20):
        assert np.array_equal(f64(Q.mxfp4_matvec(xt, w, offsets=off, out_dtype=torch.float32)), want)


@pytest.mark.parametrize("T,k,E,L,Mi", [(1, 1, 1, 32, 32), (5, 2, 3, 96, 64), (9, 4, 2, 1056, 96), (23, 3, 5, 64, 544),
                                        (7, 2, 2, 256, 1056), (6, 1, 2, 64, 3552), (4, 2, 3, 32, 4128), (3, 2, 2, 64, 8224), (1, 1, 1, 5120, 4352),
                                        (40, 32, 3, 128, 256), (100, 8, 16, 768, 512), (33, 16, 9, 1024, 768)])
def test_differences_of_close_activations(T, k, E, L, Mi):
    """Features of a token that differ by 2^-12, subtracted by the down product: they keep fp32's accuracy, in a small call
    as in a large one.

    An activation's products are sums of two terms, its functions are within 2^-20 of the value, and what
    multiplies it afterwards within 2^-22 of its block's largest, which is at most 1.1 times each; the output is rounded to bf16."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(T + k + L + Mi)
    x = np.zeros((T, L))
    x[:, 0] = r.uniform(2.0, 3.0, T)
    x[:, 1] = r.uniform(1.0, 2.0, T) * r.choice([-1, 1], T)
    x[:, L - 1] = np.abs(x[:, 1]) * 2.0 ** -12
    xt = torch.from_numpy(x).to(torch.bfloat16)
    x = f64(xt)
    gate = picks(np.zeros((E, Mi), int), L)
    up = picks(np.ones((E, Mi), int), L)
    code = r.randint(0, 8, (E, Mi)).astype(np.uint8)          # 0 to 6 times the last element
    up[0][..., -1] |= code << 4
    step = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])[code]
    p, q = r.randint(0, Mi, (E, L)), r.randint(0, Mi, (E, L))
    q = np.where(p == q, (q + 1) % Mi, q)
    out = picks(p, Mi)
    minus = picks(q, Mi, np.full(q.shape, -1))
    out = (out[0] | minus[0], out[1])
    idx = r.randint(0, E, (T, k)).astype(np.int32)
    w = np.ldexp(1.0, -r.randint(0, 4, (T, k))).astype(np.float32)
    y = f64(Q.mxfp4_experts(xt.cuda(), *cuda(idx, w), *(Q.Mxfp4(*cuda(*t)) for t in (gate, up, out))))
    want, bound = np.zeros((T, L)), np.zeros((T, L))
    for t in range(T):
        for i in range(k):
            e = idx[t, i]
            act = F.situ(x[t, 0], x[t, 1] + step[e] * x[t, L - 1], 4.0, 25.0)
            want[t] += w[t, i] * (act[p[e]] - act[q[e]])
            bound[t] += w[t, i] * 2 * (2.0 ** -20 + 1.1 * 2.0 ** -22) * np.abs(act).max()
    assert np.abs(want).max() > 50 * bound.max() / k
    bad = ~(np.abs(y - want) <= bound + 2.0 ** -8 * np.abs(want))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], y[bad][:5], want[bad][:5])


def perms(r, E, N, K):
    """Columns [E, N]: each expert's rows pick different elements, all of them where N >= K."""
    return np.stack([np.concatenate([r.permutation(K) for _ in range(-(-N // K))])[:N] for _ in range(E)])


def blocks_of(r, R, K, low, high):
    """bf16 rows with all 8 significant bits: each block's largest is a power of two between 2^-20 and 2^20, of either sign, the
    others of `low` to `high` powers less."""
    x = (1 + r.randint(0, 128, (R, K)) / 128) * np.ldexp(1.0, -r.randint(low, high + 1, (R, K)))
    top = r.randint(0, 32, (R, K // 32, 1))
    x = x.reshape(R, K // 32, 32)
    np.put_along_axis(x, top, 1.0, 2)
    size = np.ldexp(1.0, r.randint(-20, 21, (R, K // 32, 1)))
    x, size = (x * size * r.choice([-1, 1], x.shape)).reshape(R, K), np.repeat(size, 32, 2).reshape(R, K)
    return x, size


def in_pieces(n, R, elements):
    return (n + R // 8) * elements >= 1 << 26


# (rows of each expert, features, depth): a dense call, experts without rows among others, tiles of 2, 8, 16 and 24 rows
LOADS = [([600], 1000, 1024), ([300, 0, 25, 200], 1024, 1024), ([1] * 70, 1024, 1024), ([7, 0, 3, 8] * 14, 1000, 1280),
         ([16, 9, 0] * 12, 1032, 1280), ([68], 1032, 7424)]


def picked(r, loads, N, K):
    """(weights as the call takes them, offsets, what a row of each expert picks: columns and factors)."""
    import quantile_balanced_routing_gb300 as Q
    E = len(loads)
    cols, sign, e = perms(r, E, N, K), r.choice([-1, 1], (E, N)), r.randint(-20, 21, (E, N))
    c, s = picks(cols, K, sign)
    s = (s + e[..., None]).astype(np.uint8)
    off = None if E == 1 else cuda(np.concatenate([[0], np.cumsum(loads)]).astype(np.int32))[0]
    w = Q.Mxfp4(*cuda(c[0], s[0])) if E == 1 else Q.Mxfp4(*cuda(c, s))
    of = np.repeat(np.arange(E), loads)
    return w, off, cols[of], (sign * np.ldexp(1.0, e))[of]


@pytest.mark.parametrize("loads,N,K", LOADS)
def test_pieces_hold_every_digit(loads, N, K):
    """bf16 elements down to 2^-14 of their block's largest are the sum of their eight pieces, bit for bit; smaller ones are
    rounded to 2^-21 of it, ties to even (which shows that the rows did go in pieces)."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(N + K)
    R = sum(loads)
    assert in_pieces(min(len(loads), R), R, N * K)
    w, off, cols, factor = picked(r, loads, N, K)
    run = lambda x: f64(Q.mxfp4_matvec(torch.from_numpy(x).to(torch.bfloat16).cuda(), w, offsets=off, out_dtype=torch.float32))  # noqa: E731
    x, size = blocks_of(r, R, K, 1, 14)
    assert np.array_equal(run(x), np.take_along_axis(x, cols, 1) * factor)
    x, size = blocks_of(r, R, K, 15, 30)
    want = np.round(x / size * 2.0 ** 21) / 2.0 ** 21 * size
    assert (want != x).mean() > 0.5
    assert np.array_equal(run(x), np.take_along_axis(want, cols, 1) * factor)
    y = Q.mxfp4_matvec(torch.from_numpy(x).to(torch.bfloat16).cuda(), w, offsets=off)
    assert np.array_equal(f64(y), f64(torch.from_numpy(np.take_along_axis(want, cols, 1) * factor).to(torch.bfloat16)))


@pytest.mark.parametrize("loads,N,K", LOADS)
def test_pieces_hold_every_code_of_8_bits(loads, N, K):
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(N + K)
    R = sum(loads)
    w, off, cols, factor = picked(r, loads, N, K)
    codes = r.randint(0, 256, (R, K)).astype(np.uint8)
    codes[codes & 127 == 127] = 1
    scales = r.randint(60, 200, (R, K // 32)).astype(np.uint8)
    y = f64(Q.mxfp4_matvec(Q.Mxfp8(*cuda(codes, scales)), w, offsets=off, out_dtype=torch.float32))
    assert np.array_equal(y, np.take_along_axis(F.decode8(codes, scales), cols, 1) * factor)


@pytest.mark.parametrize("loads,N,K", [([8], 1000, 1024), ([3, 0, 9], 264, 544), ([2], 64, 7168), ([5, 1], 40, 8224), ([1, 2, 3] * 4, 72, 96)])
def test_small_products_hold_elements_down_to_2_32_of_the_largest(loads, N, K):
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(N + K)
    R = sum(loads)
    assert not in_pieces(min(len(loads), R), R, N * K)
    w, off, cols, factor = picked(r, loads, N, K)
    x, size = blocks_of(r, R, K, 1, 32)
    y = f64(Q.mxfp4_matvec(torch.from_numpy(x).to(torch.bfloat16).cuda(), w, offsets=off, out_dtype=torch.float32))
    assert np.array_equal(y, np.take_along_axis(x, cols, 1) * factor)


SIZES = [(1, 1, 1, 32, 32), (1, 16, 40, 512, 256), (5, 2, 3, 96, 64), (9, 4, 2, 1056, 96), (23, 3, 5, 64, 544), (30, 8, 12, 1056, 32),
         (1, 4, 6, 3584, 1024), (3, 2, 4, 64, 8224), (1, 2, 3, 8256, 64), (128, 32, 40, 64, 96), (100, 8, 16, 768, 512),
         (33, 16, 20, 1024, 768), (2, 16, 16, 2048, 1024), (260, 4, 7, 512, 512), (2, 2, 3, 64, 2048), (9, 3, 4, 96, 1600), (2, 1, 2, 32, 2080),
         (11, 3, 3, 64, 320), (3, 2, 2, 32, 4096)]


@pytest.mark.parametrize("kind", ["bf16", "mxfp8"])
@pytest.mark.parametrize("T,k,E,L,Mi", SIZES)
def test_every_route_block_and_feature_of_experts(T, k, E, L, Mi, kind):
    """Gate, up and down rows that pick one element each: an output is the sum of k activations of two elements of x,
    each within 2^-20 for the functions and 2^-22 for the split, before its rounding to bf16."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(T + k + E + L + Mi)
    x = r.uniform(0.5, 4.0, (T, L)) * r.choice([-1, 1], (T, L))
    if kind == "bf16":
        t = torch.from_numpy(x).to(torch.bfloat16).cuda()
        x = f64(t)
    else:
        codes, scales = F.quantize8(x)
        t, x = Q.Mxfp8(*cuda(codes, scales)), F.decode8(codes, scales)
    g, u, o = perms(r, E, Mi, L), perms(r, E, Mi, L), perms(r, E, L, Mi)
    sign = r.choice([-1, 1], (E, Mi))
    weights = [Q.Mxfp4(*cuda(*p)) for p in (picks(g, L), picks(u, L, sign), picks(o, Mi))]
    idx = np.stack([r.permutation(E)[:k] if k <= E else r.randint(0, E, k) for _ in range(T)]).astype(np.int32)
    if T > 4:
        idx[1], idx[2, 0], idx[3, -1] = -1, E, 1 << 30      # no route: all, one, one
    w = r.uniform(0.2, 1.0, (T, k)).astype(np.float32)
    y = f64(Q.mxfp4_experts(t, *cuda(idx, w), *weights))
    want, size = np.zeros((T, L)), np.zeros((T, L))
    for i in range(T):
        for j in range(k):
            e = idx[i, j]
            if 0 <= e < E:
                act = F.situ(x[i, g[e]], sign[e] * x[i, u[e]], 4.0, 25.0)[o[e]] * float(w[i, j])
                want[i] += act
                size[i] += np.abs(act) + 2.0 ** -2 * 16 * float(w[i, j])         # (activations are at most 16)
    bound = 2.0 ** -20 * size + (k + 2) * 2.0 ** -24 * size + 2.0 ** -8 * np.abs(want)
    bad = ~(np.abs(y - want) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], y[bad][:5], want[bad][:5])


@pytest.mark.parametrize("T,k,E,L,Mi", SIZES)
def test_experts_in_the_two_norm(T, k, E, L, Mi):
    """The distance of a token's result from the 64-bit one: the output's rounding, and three sums.

    A sum of K terms is K / 32 blocks, and at most 40 additions within a block and over the warps, each off by 2^-23 of a partial sum
    (2^-24, or a truncation); terms of random sign add up to 0.8 sqrt(K) times their result in magnitude."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(T + k + E + L + Mi)
    made = [F.weights(r, E, Mi, L), F.weights(r, E, Mi, L), F.weights(r, E, L, Mi)]
    weights = [Q.Mxfp4(*cuda(c, s)) for c, s, _ in made]
    gv, uv, ov = (v for _, _, v in made)
    idx = np.stack([r.permutation(E)[:k] if k <= E else r.randint(0, E, k) for _ in range(T)]).astype(np.int32)
    w = r.uniform(0.2, 1.0, (T, k)).astype(np.float32)
    gain = (1 + 0.3 * r.standard_normal(L)).astype(np.float32)
    rows = r.standard_normal((T, L)) * np.exp(0.5 * r.standard_normal((T, 1)))
    sums = lambda K: (K / 32 + 40) * 2.0 ** -23 * 0.8 * np.sqrt(K)  # noqa: E731
    tolerance = 2.0 ** -8 + 2.2 * sums(L) + sums(Mi) + 2.0 ** -18
    for kind in ("bf16", "mxfp8"):
        if kind == "bf16":
            t = torch.from_numpy(rows).to(torch.bfloat16).cuda()
            x = f64(t)
        else:
            codes, scales = F.quantize8(rows)
            t, x = Q.Mxfp8(*cuda(codes, scales)), F.decode8(codes, scales)
        z = np.zeros((T, L))
        for e in range(E):
            i, j = np.nonzero(idx == e)
            act = F.situ(x[i] @ gv[e].T, x[i] @ uv[e].T, 4.0, 25.0)
            np.add.at(z, i, (act @ ov[e].T) * w[i, j][:, None])
        for gamma in (None, gain):
            y = f64(Q.mxfp4_experts(t, *cuda(idx, w), *weights, gamma=None if gamma is None else cuda(gamma)[0]))
            want = z if gamma is None else F.norm(z, gamma, 1e-6)
            off = np.sqrt(((y - want) ** 2).sum(1) / (want ** 2).sum(1))
            assert (off <= tolerance).all(), (kind, gamma is None, off.max(), tolerance)


@pytest.mark.parametrize("T", [4, 64])
def test_experts_are_the_layers_routed_part(T):
    """A layer whose projections pass the first elements through and that has no shared expert, against the experts alone.

    The layer rounds activations, routes and sums to bf16 (2^-8 each, the activations' hyperbolic tangent 2^-11 more), the experts
    their output."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(T)
    d, L, E, k, Mi = 1024, 512, 64, 8, 512
    assert in_pieces(min(E, T * k), T * k, 3 * L * Mi) == (T == 64)
    made = [F.weights(r, E, Mi, L), F.weights(r, E, Mi, L), F.weights(r, E, L, Mi)]
    gate, up, out = (Q.Mxfp4(*cuda(c, s)) for c, s, _ in made)
    gain = cuda((1 + 0.3 * r.standard_normal(L)).astype(np.float32))[0]
    eye = torch.eye(L, d, device="cuda").to(torch.bfloat16)
    x = torch.from_numpy(r.standard_normal((T, d))).to(torch.bfloat16).cuda()
    layer = Q.LatentMoE(d, L, E, k, Mi, 0, expert_wfmt="mxfp4", qb_sweeps=0, max_tokens=T)
    layer.set_weights(w_router=torch.zeros(E, d, dtype=torch.bfloat16, device="cuda"), w_down=eye, w_proj_up=eye.t().contiguous(),
                      w_gate=gate.codes, s_gate=gate.scales, w_up=up.codes, s_up=up.scales, w_out=out.codes, s_out=out.scales,
                      rms_gamma=gain)
    got, routing = layer.forward(x, logits_in=cuda(r.standard_normal((T, E)).astype(np.float32))[0], want_routing=True)
    assert layer.status() == 0 and layer.uses_tensor_cores
    want = f64(Q.mxfp4_experts(x[:, :L], routing["idx"], routing["w"], gate, up, out, gamma=gain))
    got = f64(got)[:, :L]
    off = np.sqrt(((got - want) ** 2).sum(1) / (want ** 2).sum(1))
    assert (off <= 4 * 2.0 ** -8 + 2 * 2.0 ** -11).all(), off.max()
    layer.close()
