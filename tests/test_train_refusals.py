"""What the router-training and MXFP4 entry points refuse, on the host and before any device is touched (no GPU needed)."""
import pytest

import quantile_balanced_routing_gb300 as Q

torch = pytest.importorskip("torch")

FAKE = 1 << 20     # aligned fake device address: never dereferenced by the host checks
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    return Q.load_library()


def changed(args, at, value):
    a = list(args)
    a[at] = value
    return a


# T, n, k, S, dtype, logits, ld, idx, seq, mask, loss, counts, probs, tokens, workspace, bytes, stream
LOSS = [8, 16, 2, 3, 0, FAKE, 16, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, BIG, None]


@pytest.mark.parametrize("at,value", [(0, 0), (1, 1), (1, 1025), (2, 0), (2, 17), (2, 33), (3, 0), (4, 2), (5, None),
                                      (6, 15), (7, None), (8, None), (10, None), (11, None), (12, None), (13, None),
                                      (14, None), (5, FAKE + 2), (7, FAKE + 2), (14, FAKE + 16)])
def test_balance_loss_refuses(lib, at, value):
    assert lib.moe_balance_loss(*changed(LOSS, at, value)) == Q.QBMOE_EINVAL


def test_balance_workspace(lib):
    need = lib.qbmoe_balance_workspace_bytes(8, 16, 3)
    assert need > 0 and lib.qbmoe_balance_workspace_bytes(0, 16, 3) == 0
    assert lib.moe_balance_loss(*changed(LOSS, 15, need - 1)) == Q.QBMOE_EWORKSPACE


# T, n, k, S, dtype, logits, ld, idx, seq, mask, dw, dloss, counts, tokens, dlogits, ldg, stream
GRAD = [8, 16, 2, 3, 0, FAKE, 16, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2 * FAKE, 16, None]


@pytest.mark.parametrize("at,value", [(0, 0), (1, 1), (2, 0), (3, 0), (4, -1), (5, None), (6, 15), (7, None),
                                      (8, None), (11, None), (12, None), (13, None), (14, None), (15, 15),
                                      (14, 2 * FAKE + 2), (10, FAKE + 1)])
def test_router_backward_refuses(lib, at, value):
    assert lib.moe_router_backward(*changed(GRAD, at, value)) == Q.QBMOE_EINVAL


def test_router_backward_refuses_nothing_to_do_and_a_strided_alias(lib):
    a = list(GRAD)
    a[10:14] = [None] * 4
    assert lib.moe_router_backward(*a) == Q.QBMOE_EINVAL
    a = changed(GRAD, 14, FAKE)
    assert lib.moe_router_backward(*changed(a, 15, 20)) == Q.QBMOE_EINVAL


# rows, K, dtype, x, ldx, codes, scales, values, stream
QUANT = [4, 64, 1, FAKE, 64, FAKE, FAKE, FAKE, None]


@pytest.mark.parametrize("at,value", [(0, -1), (1, 0), (1, 48), (2, 2), (3, None), (3, FAKE + 8), (4, 63), (4, 68),
                                      (5, None), (5, FAKE + 8), (6, None), (7, FAKE + 8), (0, 1 << 60)])
def test_quantize_refuses(lib, at, value):
    assert lib.moe_mxfp4_quantize(*changed(QUANT, at, value)) == Q.QBMOE_EINVAL


# R, E, N, K, x_type, x, ldx, x_scales, w_codes, w_scales, offsets, y, ldy, workspace, bytes, stream
MATMUL = [4, 2, 16, 64, 2, FAKE, 64, FAKE, FAKE, FAKE, FAKE, FAKE, 16, FAKE, BIG, None]
# R, E, N, K, dy, lddy, w_codes, w_scales, offsets, dx, lddx, stream
DGRAD = [4, 2, 16, 64, FAKE, 16, FAKE, FAKE, FAKE, FAKE, 64, None]
# R, E, N, K, dy, lddy, x_codes, x_scales, offsets, dw_dtype, dw, workspace, bytes, stream
WGRAD = [4, 2, 16, 64, FAKE, 16, FAKE, FAKE, FAKE, 0, FAKE, None, 0, None]
SIZES = [(0, -1), (1, 0), (1, 1025), (2, 0), (2, 12), (3, 0), (3, 48), (3, 1 << 25)]


@pytest.mark.parametrize("at,value", SIZES + [(4, 3), (5, None), (5, FAKE + 8), (6, 72), (7, FAKE + 8),
                                              (7, None), (8, None), (9, FAKE + 8), (10, None), (10, FAKE + 4),
                                              (11, None), (12, 8), (12, 20), (12, 1 << 28), (4, 1 << 20)])
def test_matmul_refuses(lib, at, value):
    assert lib.moe_mxfp4_matmul(*changed(MATMUL, at, value)) == Q.QBMOE_EINVAL


def test_products_refuse_too_many_weight_rows(lib):
    E, N = 1024, 1 << 22
    assert lib.moe_mxfp4_matmul(*(MATMUL[:1] + [E, N] + MATMUL[3:12] + [N] + MATMUL[13:])) == Q.QBMOE_EINVAL


@pytest.mark.parametrize("x_type,ldx", [(0, 63), (0, 66), (1, 63), (1, 68), (0, 32)])
def test_matmul_refuses_rows_it_cannot_quantise(lib, x_type, ldx):
    assert lib.moe_mxfp4_matmul(*changed(changed(MATMUL, 4, x_type), 6, ldx)) == Q.QBMOE_EINVAL


@pytest.mark.parametrize("workspace", [None, FAKE + 16])
def test_matmul_needs_an_aligned_workspace_to_quantise(lib, workspace):
    assert lib.moe_mxfp4_matmul(*changed(changed(MATMUL, 4, 1), 13, workspace)) == Q.QBMOE_EINVAL


@pytest.mark.parametrize("at,value", SIZES + [(4, None), (5, 8), (5, 20), (6, None), (7, FAKE + 8), (8, None),
                                              (9, None), (10, 63), (10, 68), (10, 1 << 28)])
def test_dgrad_refuses(lib, at, value):
    assert lib.moe_mxfp4_dgrad(*changed(DGRAD, at, value)) == Q.QBMOE_EINVAL


@pytest.mark.parametrize("at,value", SIZES + [(4, None), (5, 8), (5, 20), (6, None), (7, FAKE + 8), (8, None),
                                              (9, 2), (10, None), (10, FAKE + 8), (5, 1 << 28)])
def test_wgrad_refuses(lib, at, value):
    assert lib.moe_mxfp4_wgrad(*changed(WGRAD, at, value)) == Q.QBMOE_EINVAL


def test_workspace_too_small(lib):
    need = lib.qbmoe_mxfp4_workspace_bytes(4, 64)
    assert need > 4 * 34 and lib.qbmoe_mxfp4_workspace_bytes(4, 48) == 0
    assert lib.moe_mxfp4_matmul(*changed(changed(MATMUL, 4, 1), 14, need - 1)) == Q.QBMOE_EWORKSPACE


def test_weight_gradient_workspace(lib):
    # many tiles, or few rows: none; one small matrix over many rows: its parts
    assert lib.qbmoe_mxfp4_wgrad_workspace_bytes(65536, 224, 1024, 3584) == 0
    assert lib.qbmoe_mxfp4_wgrad_workspace_bytes(300, 1, 264, 544) == 0
    need = lib.qbmoe_mxfp4_wgrad_workspace_bytes(40000, 1, 264, 544)
    assert need > 264 * 544 * 4 and need % (264 * 544 * 4) == 0
    big = [40000, 1, 264, 544, FAKE, 264, FAKE, FAKE, FAKE, 0, FAKE, FAKE, need, None]
    for at, value, code in ((11, None, Q.QBMOE_EINVAL), (11, FAKE + 8, Q.QBMOE_EINVAL), (12, need - 1, Q.QBMOE_EWORKSPACE)):
        rc = lib.moe_mxfp4_wgrad(*changed(big, at, value))
        assert rc in (code, Q.QBMOE_ECUDA, Q.QBMOE_EARCH)    # without a GPU the device is asked first


def refuses(fn, *args, **kw):
    with pytest.raises(Q.QbmoeError) as e:
        fn(*args, **kw)
    assert e.value.code == Q.QBMOE_EINVAL
    return str(e.value)


def test_python_refuses_wrong_tensors():
    x, idx = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    assert "current CUDA device" in refuses(Q.balance_loss, x, idx)
    refuses(Q.balance_loss, x.double(), idx)
    refuses(Q.balance_loss, x.t(), idx)
    refuses(Q.balance_loss, x, idx.long())
    refuses(Q.balance_loss, x, idx[:3])
    refuses(Q.balance_loss, x, idx, seq_offsets=torch.zeros(3, dtype=torch.int64))
    refuses(Q.balance_loss, x, idx, token_mask=torch.ones(3, dtype=torch.bool))
    refuses(Q.router_backward, x, idx)
    refuses(Q.router_backward, x, idx, dloss=torch.ones(1))
    refuses(Q.router_backward, x, idx, dw=torch.zeros(4, 3))
    refuses(Q.router_backward, x, idx, dw=torch.zeros(4, 2), out=torch.zeros(4, 8, dtype=torch.bfloat16))
    refuses(Q.mxfp4_quantize, torch.zeros(4, 40))
    refuses(Q.mxfp4_quantize, torch.zeros(4, 64).half())
    refuses(Q.mxfp4_quantize, torch.zeros(64, 4).t())
    refuses(Q.mxfp4_quantize, torch.zeros(4, 66)[:, :64])      # rows off 16-byte boundaries
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    xq, w, wg = Q.Mxfp4(u8(4, 32), u8(4, 2)), Q.Mxfp4(u8(16, 32), u8(16, 2)), Q.Mxfp4(u8(3, 16, 32), u8(3, 16, 2))
    off = torch.zeros(4, dtype=torch.int32)
    assert "current CUDA device" in refuses(Q.mxfp4_matmul, xq, w)
    refuses(Q.mxfp4_matmul, xq, (u8(16, 32), u8(16, 2)))
    refuses(Q.mxfp4_matmul, xq, Q.Mxfp4(u8(16, 48), u8(16, 3)))      # another K
    refuses(Q.mxfp4_matmul, xq, Q.Mxfp4(u8(12, 32), u8(12, 2)))
    refuses(Q.mxfp4_matmul, torch.zeros(4, 64).half(), w)
    refuses(Q.mxfp4_matmul, xq, wg)
    refuses(Q.mxfp4_matmul, xq, wg, off[:3])
    refuses(Q.mxfp4_matmul, xq, wg, off.long())
    refuses(Q.Mxfp4, u8(4, 32), u8(4, 3))
    refuses(Q.Mxfp4, u8(4, 32), u8(5, 2))
    refuses(Q.Mxfp4, u8(4, 24), u8(4, 1))
    refuses(Q.Mxfp4, u8(4, 32).int(), u8(4, 2))
    refuses(Q.Mxfp4, u8(32, 4).t(), u8(4, 2))
    dy = torch.zeros(4, 16, dtype=torch.bfloat16)
    refuses(Q.mxfp4_matmul_backward, dy.float(), xq, w)
    refuses(Q.mxfp4_matmul_backward, dy[:3], xq, w)
    refuses(Q.mxfp4_matmul_backward, dy, xq, w, dw_dtype=torch.float16)
    refuses(Q.mxfp4_matmul_backward, dy, (xq.codes, xq.scales), w)
    refuses(Q.mxfp4_matmul_backward, dy, xq, wg)
