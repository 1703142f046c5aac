"""The norm's and the few-row calls' formulas against differences, and what the calls refuse, on the host (no GPU needed)."""
import numpy as np
import pytest

import few_rows_reference as F
import quantile_balanced_routing_gb300 as Q

torch = pytest.importorskip("torch")

FAKE, BIG = 1 << 20, 1 << 40      # aligned fake device address: never dereferenced by the host checks
MOST = (1 << 31) - (1 << 24)


@pytest.fixture(scope="module")
def lib():
    return Q.load_library()


def changed(args, at, value):
    a = list(args)
    a[at] = value
    return a


@pytest.mark.parametrize("with_total", [False, True])
def test_the_norms_gradient_is_that_of_differences(with_total):
    r = np.random.RandomState(0)
    T, H, eps = 4, 24, 1e-3
    v, dn, g = r.standard_normal((T, H)), r.standard_normal((T, H)), 1 + 0.3 * r.standard_normal(H)
    do = r.standard_normal((T, H)) if with_total else None
    loss = lambda v, g: (dn * F.norm(v, g, eps)).sum() + (0.0 if do is None else (do * v).sum())  # noqa: E731
    (dx, _), (dg, _) = F.norm_backward(dn, v, g, do, eps)
    h = 1e-6
    for _ in range(5):
        a, b = r.standard_normal((T, H)), r.standard_normal(H)
        slope = (loss(v + h * a, g + h * b) - loss(v - h * a, g - h * b)) / (2 * h)
        assert abs(slope - (dx * a).sum() - (dg * b).sum()) < 1e-7 * (1 + np.abs(dx).sum())


def test_the_references_eight_bit_grid():
    assert F.E4M3[126] == 448 and F.E4M3[1] == 2.0 ** -9 and F.E4M3[56] == 1.0 and len(F.E4M3) == 127
    x = np.random.RandomState(1).standard_normal((5, 96))
    c, s = F.quantize8(x)
    t = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy() * np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, 1)
    assert np.array_equal(t, F.decode8(c, s)) and np.abs(t - x).max() <= 2.0 ** -4 * np.abs(x).max()


# T, H, x_type, x, ldx, res_type, residual, ldr, gamma, eps, total, ldt, y, ldy, codes, scales, stream
NORM = [4, 64, 1, FAKE, 64, 0, FAKE, 64, FAKE, 1e-6, FAKE, 64, FAKE, 64, FAKE, FAKE, None]


@pytest.mark.parametrize("at,value", [(0, -1), (0, MOST + 1), (1, 0), (1, 48), (1, 16385), (2, 2), (2, 3), (3, None), (3, FAKE + 1),
                                      (4, 63), (5, 2), (6, None), (6, FAKE + 2), (7, 63), (8, None), (8, FAKE + 2),
                                      (9, -1.0), (9, float("nan")), (9, float("inf")), (10, None), (10, FAKE + 2), (11, 63),
                                      (12, FAKE + 1), (13, 63), (14, None), (14, FAKE + 4), (15, None)])
def test_add_rmsnorm_refuses(lib, at, value):
    assert lib.moe_add_rmsnorm(*changed(NORM, at, value)) == Q.QBMOE_EINVAL


def test_add_rmsnorm_refuses_a_call_without_outputs(lib):
    assert lib.moe_add_rmsnorm(*(NORM[:12] + [None, 0, None, None, None])) == Q.QBMOE_EINVAL


# T, H, dn_type, dn, lddn, total_type, total, ldt, gamma, eps, dtotal, lddt, dx, lddx, dgamma, workspace, bytes, stream
BACK = [4, 64, 1, FAKE, 64, 0, FAKE, 64, FAKE, 1e-6, FAKE, 64, FAKE, 64, FAKE, FAKE, BIG, None]


@pytest.mark.parametrize("at,value", [(0, -1), (0, MOST + 1), (1, 0), (1, 16385), (2, 2), (3, None), (3, FAKE + 1), (4, 63),
                                      (5, 3), (6, None), (6, FAKE + 2), (7, 63), (8, None), (8, FAKE + 1), (9, -1.0),
                                      (10, FAKE + 2), (11, 63), (12, None), (12, FAKE + 2), (13, 63), (14, FAKE + 2),
                                      (15, None), (15, FAKE + 16)])
def test_add_rmsnorm_backward_refuses(lib, at, value):
    assert lib.moe_add_rmsnorm_backward(*changed(BACK, at, value)) == Q.QBMOE_EINVAL


def test_add_rmsnorm_backward_workspace(lib):
    need = lib.qbmoe_add_rmsnorm_workspace_bytes(4, 64)
    assert need >= 256 and lib.qbmoe_add_rmsnorm_workspace_bytes(4, 0) == 0 < lib.qbmoe_add_rmsnorm_workspace_bytes(MOST, 16384)
    assert lib.moe_add_rmsnorm_backward(*changed(BACK, 16, need - 1)) == Q.QBMOE_EWORKSPACE


# R, E, N, K, x_type, x, ldx, x_scales, w_codes, w_scales, offsets, y_type, y, ldy, workspace, bytes, stream
MATVEC = [4, 2, 16, 64, 3, FAKE, 64, FAKE, FAKE, FAKE, FAKE, 1, FAKE, 16, None, 0, None]


@pytest.mark.parametrize("at,value", [(0, -1), (0, MOST + 1), (1, 0), (1, 1025), (2, 0), (2, 12), (2, (1 << 24) + 8), (3, 0), (3, 48),
                                      (3, 65568), (4, 0), (4, 2), (4, 4), (5, None), (5, FAKE + 8), (6, 72), (7, None),
                                      (7, FAKE + 8), (8, None), (8, FAKE + 8), (9, None), (9, FAKE + 8), (10, None), (10, FAKE + 2),
                                      (11, 2), (11, 3), (12, None), (12, FAKE + 1), (13, 15)])
def test_matvec_refuses(lib, at, value):
    assert lib.moe_mxfp4_matvec(*changed(MATVEC, at, value)) == Q.QBMOE_EINVAL


@pytest.mark.parametrize("ldx", [63, 68, 32])
def test_matvec_refuses_strides_off_16_bytes(lib, ldx):
    assert lib.moe_mxfp4_matvec(*changed(changed(MATVEC, 4, 1), 6, ldx)) == Q.QBMOE_EINVAL


def test_matvec_workspace(lib):
    assert lib.qbmoe_mxfp4_matvec_workspace_bytes(100, 64, 8192) == 0
    assert lib.qbmoe_mxfp4_matvec_workspace_bytes(100, 4096, 8192) >= 100 * 8 * (4096 + 256)   # in pieces
    need = lib.qbmoe_mxfp4_matvec_workspace_bytes(4, 16, 16384)
    if need:
        big = changed(changed(changed(MATVEC, 3, 16384), 6, 16384), 15, BIG)
        for ws in (None, FAKE + 16):
            assert lib.moe_mxfp4_matvec(*changed(big, 14, ws)) == Q.QBMOE_EINVAL
        assert lib.moe_mxfp4_matvec(*changed(changed(big, 14, FAKE), 15, need - 1)) == Q.QBMOE_EWORKSPACE


# T, k, E, L, M, x_type, x, ldx, x_scales, idx, w, gate, gate_s, up, up_s, out, out_s, beta1, beta2, gamma, eps, y, ldy, ws, bytes, stream
EXPERTS = [4, 2, 8, 64, 96, 3, FAKE, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4.0, 25.0, FAKE, 1e-6, FAKE, 64,
           FAKE, BIG, None]


@pytest.mark.parametrize("at,value", [(0, -1), (0, 2049), (1, 0), (1, 33), (2, 0), (2, 1025), (3, 48), (3, 65568), (4, 0), (4, 48),
                                      (4, 65568), (5, 0), (5, 2), (6, None), (6, FAKE + 8), (7, 72), (8, None), (8, FAKE + 8),
                                      (9, None), (9, FAKE + 2), (10, None), (10, FAKE + 2), (11, None), (11, FAKE + 8), (12, FAKE + 8),
                                      (13, None), (14, None), (15, FAKE + 8), (16, None), (17, 0.0), (17, float("nan")),
                                      (18, -1.0), (19, FAKE + 2), (20, -1.0), (20, float("nan")), (21, None), (21, FAKE + 1),
                                      (22, 63), (23, None), (23, FAKE + 16)])
def test_experts_refuses(lib, at, value):
    assert lib.moe_mxfp4_experts(*changed(EXPERTS, at, value)) == Q.QBMOE_EINVAL


def test_experts_workspace(lib):
    need = lib.qbmoe_mxfp4_experts_workspace_bytes(4, 2, 64, 96)
    assert need > 0 and lib.qbmoe_mxfp4_experts_workspace_bytes(2049, 2, 64, 96) == 0
    assert lib.moe_mxfp4_experts(*changed(EXPERTS, 24, need - 1)) == Q.QBMOE_EWORKSPACE


def refuses(fn, *args, **kw):
    with pytest.raises(Q.QbmoeError) as e:
        fn(*args, **kw)
    assert e.value.code == Q.QBMOE_EINVAL
    return str(e.value)


def test_python_refuses_wrong_tensors():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    x, g = torch.zeros(4, 64), torch.ones(64)
    assert "current CUDA device" in refuses(Q.add_rmsnorm, x, g)
    refuses(Q.add_rmsnorm, x.half(), g)
    refuses(Q.add_rmsnorm, x, g.double())
    refuses(Q.add_rmsnorm, x, g[:32])
    refuses(Q.add_rmsnorm, x, torch.ones(128)[::2])
    refuses(Q.add_rmsnorm, torch.zeros(64, 4).t(), g)
    refuses(Q.add_rmsnorm, torch.zeros(2, 4, 128)[..., ::2], g)
    refuses(Q.add_rmsnorm, x, g, residual=x[:3])
    refuses(Q.add_rmsnorm, x, g, residual=x.half())
    refuses(Q.add_rmsnorm, x, g, total=x)
    refuses(Q.add_rmsnorm, x, g, residual=x, total=x.bfloat16())
    refuses(Q.add_rmsnorm, x, g, eps=-1.0)
    refuses(Q.add_rmsnorm, x, g, eps=float("nan"))
    refuses(Q.add_rmsnorm, torch.zeros(4, 48), torch.ones(48), mxfp8=True)
    refuses(Q.add_rmsnorm, torch.zeros(()), g)
    refuses(Q.add_rmsnorm_backward, x, x[:3], g)
    refuses(Q.add_rmsnorm_backward, x.half(), x, g)
    refuses(Q.add_rmsnorm_backward, x, x, g, dtotal=x.bfloat16())
    assert "current CUDA device" in refuses(Q.add_rmsnorm_backward, x, x, g)
    refuses(Q.Mxfp8, u8(4, 64), u8(4, 3))
    refuses(Q.Mxfp8, u8(4, 48), u8(4, 1))
    refuses(Q.Mxfp8, u8(4, 64).float(), u8(4, 2))
    refuses(Q.Mxfp8, u8(64, 4).t(), u8(4, 2))
    refuses(Q.Mxfp8, u8(4, 64), u8(5, 2))
    x8, xb = Q.Mxfp8(u8(4, 64), u8(4, 2)), x.bfloat16()
    w, wg, off = Q.Mxfp4(u8(16, 32), u8(16, 2)), Q.Mxfp4(u8(3, 16, 32), u8(3, 16, 2)), torch.zeros(4, dtype=torch.int32)
    assert "current CUDA device" in refuses(Q.mxfp4_matvec, xb, w)
    refuses(Q.mxfp4_matvec, x, w)
    refuses(Q.mxfp4_matvec, xb, w, out_dtype=torch.float16)
    refuses(Q.mxfp4_matvec, xb[:, :32], w)
    refuses(Q.mxfp4_matvec, xb[0], w)
    refuses(Q.mxfp4_matvec, x8, (w.codes, w.scales))
    refuses(Q.mxfp4_matvec, x8, wg)
    refuses(Q.mxfp4_matvec, x8, wg, off.long())
    refuses(Q.mxfp4_matvec, x8, Q.Mxfp4(u8(12, 32), u8(12, 2)))
    refuses(Q.mxfp4_matvec, torch.zeros(4, 66, dtype=torch.bfloat16)[:, 2:], w)
    idx, m = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    gate, out = Q.Mxfp4(u8(3, 96, 32), u8(3, 96, 2)), Q.Mxfp4(u8(3, 64, 48), u8(3, 64, 3))
    ok = [x8, idx, m, gate, gate, out]
    assert "current CUDA device" in refuses(Q.mxfp4_experts, *ok)
    for at, value in ((0, x), (0, xb[:3]), (1, idx.long()), (1, idx[:3]), (1, torch.zeros(4, 33, dtype=torch.int32)), (2, m.double()),
                      (2, m[:3]), (3, w), (3, (gate.codes, gate.scales)), (4, out), (5, gate)):
        refuses(Q.mxfp4_experts, *changed(ok, at, value))
    refuses(Q.mxfp4_experts, *ok, gamma=torch.ones(96))
    refuses(Q.mxfp4_experts, *ok, gamma=torch.ones(64).double())
    refuses(Q.mxfp4_experts, *ok, eps=-1.0)
    refuses(Q.mxfp4_experts, *ok, beta1=0.0)
    refuses(Q.mxfp4_experts, *ok, beta2=float("inf"))


def test_python_refuses_sizes_that_c_cannot_hold():
    """Tensors without storage: a size of 2^32 + 32 must not reach the library as 32."""
    new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="meta")  # noqa: E731
    u8 = lambda *s: new(*s, dtype=torch.uint8)  # noqa: E731
    f32 = lambda *s: new(*s, dtype=torch.float32)  # noqa: E731
    i32 = lambda *s: new(*s, dtype=torch.int32)  # noqa: E731
    wrap = (1 << 32) + 32
    one = Q.Mxfp4(u8(8, 16), u8(8, 1))
    exp = lambda E, M, L: Q.Mxfp4(u8(E, M, L // 2), u8(E, M, L // 32))  # noqa: E731
    calls = [
        lambda: Q.add_rmsnorm(new(wrap, 32), f32(32)),
        lambda: Q.add_rmsnorm(new(2, wrap, 32), f32(32)),
        lambda: Q.add_rmsnorm_backward(new(wrap, 32), new(wrap, 32), f32(32)),
        lambda: Q.mxfp4_matvec(new(wrap, 32), one),
        lambda: Q.mxfp4_matvec(Q.Mxfp8(u8(wrap, 32), u8(wrap, 1)), one),
        lambda: Q.mxfp4_matvec(new(4, 65568), Q.Mxfp4(u8(8, 32784), u8(8, 2049))),
        lambda: Q.mxfp4_matvec(new(4, 32), Q.Mxfp4(u8(wrap, 16), u8(wrap, 1))),
        lambda: Q.mxfp4_experts(new(wrap, 32), i32(wrap, 2), f32(wrap, 2), exp(2, 32, 32), exp(2, 32, 32), exp(2, 32, 32)),
        lambda: Q.mxfp4_experts(new(2049, 32), i32(2049, 2), f32(2049, 2), exp(2, 32, 32), exp(2, 32, 32), exp(2, 32, 32)),
        lambda: Q.mxfp4_experts(new(4, 32), i32(4, 2), f32(4, 2), exp(2, wrap, 32), exp(2, wrap, 32), exp(2, 32, wrap)),
    ]
    for call in calls:
        with pytest.raises(Q.QbmoeError, match="at most") as e:
            call()
        assert e.value.code == Q.QBMOE_EINVAL
    with pytest.raises(Q.QbmoeError, match="1 to 16384"):
        Q.add_rmsnorm(new(4, wrap), f32(wrap))
