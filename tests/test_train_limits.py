"""Limits of the router-training and MXFP4 calls, checked on the host (no GPU needed)."""
import ctypes

import pytest

import quantile_balanced_routing_gb300 as Q

torch = pytest.importorskip("torch")


def closed_layer():
    lay = object.__new__(Q.LatentMoE)
    lay.lib, lay.ctx = Q.load_library(), ctypes.c_void_p()
    return lay


def test_hooks_of_a_closed_layer_are_refused():
    lay = closed_layer()
    try:
        assert lay.set_wait_limit(200) == Q.QBMOE_EINVAL
        assert lay.debug_stall(True) == Q.QBMOE_EINVAL
    finally:
        lay.lib.qbmoe_set_wait_limit(None, 0)
        lay.lib.qbmoe_debug_stall(None, 0)


FAKE, BIG = 1 << 20, 1 << 40      # never dereferenced: the sizes are refused first
MOST = (1 << 31) - (1 << 24)      # tokens, sequences or rows: sizes rounded up to tiles stay in 32 bits


@pytest.mark.parametrize("T,S", [(MOST + 1, 1), ((1 << 31) - 1, 1), (8, MOST + 1)])
def test_tokens_and_sequences_past_32_bits_of_tiles(T, S):
    lib = Q.load_library()
    assert lib.qbmoe_balance_workspace_bytes(T, 2, S) == 0 < lib.qbmoe_balance_workspace_bytes(MOST, 2, 1)
    assert lib.moe_balance_loss(T, 2, 1, S, 1, FAKE, 2, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 60,
                                None) == Q.QBMOE_EINVAL
    assert lib.moe_router_backward(T, 2, 1, S, 1, FAKE, 2, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, 2 * FAKE, 2,
                                   None) == Q.QBMOE_EINVAL


@pytest.mark.parametrize("R", [MOST + 1, (1 << 31) - 1])
def test_rows_past_32_bits_of_tiles(R):
    lib = Q.load_library()
    assert lib.qbmoe_mxfp4_workspace_bytes(R, 32) == 0 < lib.qbmoe_mxfp4_workspace_bytes(MOST, 32)
    assert lib.qbmoe_mxfp4_wgrad_workspace_bytes(R, 1, 8, 32) == 0 < lib.qbmoe_mxfp4_wgrad_workspace_bytes(MOST, 1, 8, 32)
    assert lib.moe_mxfp4_matmul(R, 1, 8, 32, 2, FAKE, 32, FAKE, FAKE, FAKE, None, FAKE, 8, None, 0,
                                None) == Q.QBMOE_EINVAL
    assert lib.moe_mxfp4_dgrad(R, 1, 8, 32, FAKE, 8, FAKE, FAKE, None, FAKE, 32, None) == Q.QBMOE_EINVAL
    assert lib.moe_mxfp4_wgrad(R, 1, 8, 32, FAKE, 8, FAKE, FAKE, None, 1, FAKE, FAKE, BIG, None) == Q.QBMOE_EINVAL


def test_python_refuses_sizes_that_c_cannot_hold():
    """Tensors without storage: a size of 2^32 + 32 must not reach the library as 32."""
    new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="meta")  # noqa: E731
    u8 = lambda *s: new(*s, dtype=torch.uint8)  # noqa: E731
    i32 = lambda *s: new(*s, dtype=torch.int32)  # noqa: E731
    wrap = (1 << 32) + 32
    one = Q.Mxfp4(u8(8, 16), u8(8, 1))
    calls = [
        lambda: Q.balance_loss(new(wrap, 8), i32(wrap, 2)),
        lambda: Q.balance_loss(new(4, 8), i32(4, 2), seq_offsets=i32(wrap + 1)),
        lambda: Q.router_backward(new(wrap, 8), i32(wrap, 2), dw=new(wrap, 2, dtype=torch.float32)),
        lambda: Q.mxfp4_quantize(new(1, wrap)),
        lambda: Q.mxfp4_quantize(new(1 << 36, 32)),
        lambda: Q.mxfp4_matmul(new(wrap, 32), one),
        lambda: Q.mxfp4_matmul(Q.Mxfp4(u8(wrap, 16), u8(wrap, 1)), one),
        lambda: Q.mxfp4_matmul(new(4, 32), Q.Mxfp4(u8(wrap, 16), u8(wrap, 1))),
        lambda: Q.mxfp4_matmul(new(4, wrap), Q.Mxfp4(u8(8, wrap // 2), u8(8, wrap // 32))),
        lambda: Q.mxfp4_matmul(new(4, 32), Q.Mxfp4(u8(1024, 1 << 22, 16), u8(1024, 1 << 22, 1)), i32(1025)),
        lambda: Q.mxfp4_matmul_backward(new(wrap, 8), Q.Mxfp4(u8(wrap, 16), u8(wrap, 1)), one),
        lambda: Q.mxfp4_matmul_backward(torch.empty_strided((4, 8), (1 << 28, 1), dtype=torch.bfloat16, device="meta"),
                                        Q.Mxfp4(u8(4, 16), u8(4, 1)), one),
    ]
    for call in calls:
        with pytest.raises(Q.QbmoeError, match="at most") as e:
            call()
        assert e.value.code == Q.QBMOE_EINVAL


def test_any_number_of_sequences_up_to_the_limit_has_a_workspace():
    lib = Q.load_library()
    for S in (65535, 65536, 1 << 20, MOST):
        assert lib.qbmoe_balance_workspace_bytes(8, 2, S) > 16 * S


def test_weight_gradient_refuses_its_workspace_on_the_host():
    """One small matrix over many rows needs a workspace; a wrong one is refused before any device is touched."""
    lib = Q.load_library()
    need = lib.qbmoe_mxfp4_wgrad_workspace_bytes(40000, 1, 264, 544)
    call = lambda ws, size: lib.moe_mxfp4_wgrad(40000, 1, 264, 544, FAKE, 264, FAKE, FAKE, None, 0, FAKE, ws, size,  # noqa: E731
                                                None)
    assert need > 0
    assert call(None, need) == Q.QBMOE_EINVAL
    assert call(FAKE + 8, need) == Q.QBMOE_EINVAL
    assert call(FAKE, need - 1) == Q.QBMOE_EWORKSPACE


def test_python_names_what_is_off_a_16_byte_boundary():
    def off(dtype, *shape):
        size = 1
        for s in shape:
            size *= s
        return torch.zeros(size + 1, dtype=dtype)[1:].view(shape)

    bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    w, x = (Q.Mxfp4(torch.zeros(r, 32, dtype=u8), torch.zeros(r, 2, dtype=u8)) for r in (16, 4))
    bad = Q.Mxfp4(off(u8, 16, 32), w.scales)
    dy = torch.zeros(4, 16, dtype=bf16)
    calls = [
        lambda: Q.mxfp4_quantize(off(bf16, 4, 64)),
        lambda: Q.mxfp4_quantize(off(f32, 4, 64)),
        lambda: Q.mxfp4_matmul(off(bf16, 4, 64), w),
        lambda: Q.mxfp4_matmul(x, bad),
        lambda: Q.mxfp4_matmul(bad, w),
        lambda: Q.mxfp4_matmul_backward(off(bf16, 4, 16), x, w),
        lambda: Q.mxfp4_matmul_backward(dy, x, bad),
        lambda: Q.mxfp4_matmul_backward(torch.zeros(16, 16, dtype=bf16), bad, w),
    ]
    for call in calls:
        with pytest.raises(Q.QbmoeError, match="16-byte boundary") as e:
            call()
        assert e.value.code == Q.QBMOE_EINVAL
