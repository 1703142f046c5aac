"""Waits of the few-row products that run out end their kernels, and are reported."""
import numpy as np
import pytest

import few_rows_reference as F

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def weights(r, *shape):
    import quantile_balanced_routing_gb300 as Q
    c, s, _ = F.weights(r, *shape)
    return Q.Mxfp4(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda())


@pytest.mark.parametrize("R,N,K", [(3, 40, 96), (5, 72, 1024), (9, 64, 3584), (2, 64, 7168), (2, 16, 8448), (1000, 648, 1024)])
def test_product(R, N, K):
    import quantile_balanced_routing_gb300 as Q
    lib = Q.load_library()
    w = weights(np.random.RandomState(0), N, K)
    x = torch.randn(R, K, device="cuda").to(torch.bfloat16)
    want = Q.mxfp4_matvec(x, w)
    Q.qbmoe_status(None, None)
    try:
        assert lib.qbmoe_set_wait_limit(None, 200) == 0 and lib.qbmoe_debug_stall(None, 1) == 0
        Q.mxfp4_matvec(x, w)
    finally:
        lib.qbmoe_set_wait_limit(None, 0), lib.qbmoe_debug_stall(None, 0)
    assert Q.qbmoe_status(None, None) == Q.QBMOE_ETIMEOUT
    assert torch.equal(Q.mxfp4_matvec(x, w), want) and Q.qbmoe_status(None, None) == 0


@pytest.mark.parametrize("T,k,E,L,Mi", [(3, 2, 4, 96, 64), (5, 4, 9, 2048, 512), (100, 8, 16, 768, 512)])
def test_experts(T, k, E, L, Mi):
    import quantile_balanced_routing_gb300 as Q
    lib = Q.load_library()
    r = np.random.RandomState(1)
    g, u, o = weights(r, E, Mi, L), weights(r, E, Mi, L), weights(r, E, L, Mi)
    x = torch.randn(T, L, device="cuda").to(torch.bfloat16)
    idx = torch.from_numpy(r.randint(0, E, (T, k)).astype(np.int32)).cuda()
    w = torch.rand(T, k, device="cuda")
    want = Q.mxfp4_experts(x, idx, w, g, u, o)
    Q.qbmoe_status(None, None)
    try:
        assert lib.qbmoe_set_wait_limit(None, 200) == 0 and lib.qbmoe_debug_stall(None, 1) == 0
        Q.mxfp4_experts(x, idx, w, g, u, o)
    finally:
        lib.qbmoe_set_wait_limit(None, 0), lib.qbmoe_debug_stall(None, 0)
    assert Q.qbmoe_status(None, None) == Q.QBMOE_ETIMEOUT
    assert torch.equal(Q.mxfp4_experts(x, idx, w, g, u, o), want) and Q.qbmoe_status(None, None) == 0
