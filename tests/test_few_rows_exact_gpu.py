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
