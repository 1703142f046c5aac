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
