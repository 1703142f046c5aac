"""The norm's and the few-row calls at the edges of what they take: in place, the largest counts, tensors beyond 2^32 bytes,
captured as a process's first call of them, by two host threads at once."""
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest

import few_rows_reference as F

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def stream():
    return torch.cuda.current_stream().cuda_stream or None


def kind(t):
    return 0 if t.dtype is torch.float32 else 1


def norm(x, gamma, residual, total, y):
    import quantile_balanced_routing_gb300 as Q
    T, H = x.shape
    at = lambda t: (None, 0) if t is None else (t.data_ptr(), t.stride(0))  # noqa: E731
    rp, rs = at(residual)
    tp, ts = at(total)
    return Q.load_library().moe_add_rmsnorm(T, H, kind(x), *at(x), 0 if residual is None else kind(residual), rp, rs, gamma.data_ptr(),
                                            1e-6, tp, ts, *at(y), None, None, stream())


def backward(dn, total, gamma, dtotal, dx, dgamma):
    import quantile_balanced_routing_gb300 as Q
    T, H = total.shape
    lib = Q.load_library()
    need = lib.qbmoe_add_rmsnorm_workspace_bytes(T, H)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    return lib.moe_add_rmsnorm_backward(T, H, kind(dn), dn.data_ptr(), dn.stride(0), kind(total), total.data_ptr(), total.stride(0),
                                        gamma.data_ptr(), 1e-6, None if dtotal is None else dtotal.data_ptr(),
                                        0 if dtotal is None else dtotal.stride(0), dx.data_ptr(), dx.stride(0), dgamma.data_ptr(),
                                        ws.data_ptr(), need, stream())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H", [(5, 33), (40, 1000), (9, 2021), (3, 7168), (1700, 1056), (700, 7168), (400, 8448)])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 80])
def test_in_place(T, H, dtype, size):
    """total in the residual or in x; dx in dtotal or in dn, also of rows that are scaled first: the same bits as elsewhere."""
    new = lambda s: (size * torch.randn(T, H + 8, device="cuda", generator=torch.Generator("cuda").manual_seed(s))).to(dtype)[:, :H]  # noqa: E731
    x, r, d, o = new(0), new(1), new(2), new(3)
    g = 1 + 0.1 * torch.randn(H, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    total, y = torch.empty_like(x), torch.empty_like(x)
    assert norm(x, g, r, total, y) == 0
    for where in ("residual", "x"):
        x1, r1, y1 = (t.clone(memory_format=torch.preserve_format) for t in (x, r, y))
        into = r1 if where == "residual" else x1
        assert norm(x1, g, r1, into, y1) == 0
        assert torch.equal(into, total) and torch.equal(y1, y)
    dx, dg, dg1 = torch.empty_like(x), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    assert backward(d, total, g, o, dx, dg) == 0
    for where in ("dtotal", "dn"):
        d1, o1 = (t.clone(memory_format=torch.preserve_format) for t in (d, o))
        into = o1 if where == "dtotal" else d1
        assert backward(d1, total, g, o1, into, dg1) == 0
        assert torch.equal(into, dx) and torch.equal(dg1, dg)


def weights(r, *shape):
    import quantile_balanced_routing_gb300 as Q
    c, s, v = F.weights(r, *shape)
    return Q.Mxfp4(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()), v


@pytest.mark.parametrize("L,Mi", [(32, 64), (256, 256)])
def test_the_most_experts_and_routes(L, Mi):
    """1024 experts, 4096 routes, 32 a token, each expert four times: both ways to form the products."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(L)
    T, k, E = 128, 32, 1024
    (g, gv), (u, uv), (o, ov) = weights(r, E, Mi, L), weights(r, E, Mi, L), weights(r, E, L, Mi)
    idx = np.concatenate([r.permutation(E) for _ in range(4)]).reshape(T, k).astype(np.int32)
    w = r.uniform(0.2, 1.0, (T, k)).astype(np.float32)
    x = torch.from_numpy(r.standard_normal((T, L))).to(torch.bfloat16).cuda()
    y = Q.mxfp4_experts(x, torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), g, u, o).double().cpu().numpy()
    xv = x.double().cpu().numpy()
    want = np.zeros((T, L))
    for e in range(E):
        i, j = np.nonzero(idx == e)
        np.add.at(want, i, (F.situ(xv[i] @ gv[e].T, xv[i] @ uv[e].T, 4.0, 25.0) @ ov[e].T) * w[i, j][:, None])
    off = np.sqrt(((y - want) ** 2).sum(1) / (want ** 2).sum(1))
    # the output's rounding; sums of 256 terms or fewer (48 additions deep, 13 times their result in magnitude); 32 routes
    assert (off <= 2.0 ** -8 + 3.2 * 48 * 13 * 2.0 ** -23 + 40 * 2.0 ** -24).all(), off.max()
    off = torch.arange(0, 4097, 4, dtype=torch.int32, device="cuda")
    rows = torch.from_numpy(r.standard_normal((4096, L))).to(torch.bfloat16).cuda()
    y = Q.mxfp4_matvec(rows, g, offsets=off, out_dtype=torch.float32).double().cpu().numpy().reshape(E, 4, Mi)
    want = np.einsum("erk,emk->erm", rows.double().cpu().numpy().reshape(E, 4, L), gv)
    assert (np.abs(y - want).max(2) <= (48 * 13 * 2.0 ** -23 + 2.0 ** -20) * np.abs(want).max(2)).all()


@pytest.mark.parametrize("E,N,K", [(40, 65536, 4096), (1024, 1024, 16384)])
def test_weights_beyond_4_gb(E, N, K):
    """The first, a middle and the last expert of weights whose bytes and elements pass 2^32: in pieces, and in slabs of the depth."""
    import quantile_balanced_routing_gb300 as Q
    g = torch.Generator("cuda").manual_seed(E)
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(118, 122, (E, N, K // 32), dtype=torch.uint8, device="cuda", generator=g)
    assert codes.numel() > 1 << 32
    x = torch.randn(7, K, device="cuda", generator=g).to(torch.bfloat16)
    of = [0, E // 2 + 1, E - 1]
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[of[0] + 1:], off[of[1] + 1:], off[of[2] + 1:] = 2, 3, 7
    y = Q.mxfp4_matvec(x, Q.Mxfp4(codes, scales), offsets=off.cuda(), out_dtype=torch.float32).double()
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    grid = torch.cat((grid, -grid))
    for e, lo, hi in zip(of, (0, 2, 3), (2, 3, 7)):
        w = torch.stack((grid[(codes[e] & 15).int()], grid[(codes[e] >> 4).int()]), -1).flatten(-2)
        w *= torch.exp2(scales[e].double() - 127).repeat_interleave(32, -1)
        want = x[lo:hi].double() @ w.T
        size = x[lo:hi].double().norm(dim=1)[:, None] * w.norm(dim=1)[None]
        # K / 32 + 40 additions, each 2^-23 of a partial sum, and the split's 2^-22 of each block's largest (about 2.5 times its elements)
        assert ((y[lo:hi] - want).abs() <= ((K / 32 + 40) * 2.0 ** -23 + 2.5 * 2.0 ** -22) * size).all()
    assert Q.qbmoe_status(None, None) == 0


def test_a_norm_beyond_2_32_elements():
    import quantile_balanced_routing_gb300 as Q
    T, H = (1 << 18) + 5, 16384
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    part = torch.randn(1024, H, device="cuda", generator=torch.Generator("cuda").manual_seed(0)).to(torch.bfloat16)
    for i in range(0, T, 1024):
        x[i:i + 1024] = part[:T - i]
    g = torch.ones(H, device="cuda")
    r = Q.add_rmsnorm(x, g, mxfp8=True)
    few = Q.add_rmsnorm(part, g, mxfp8=True)
    for i in (0, T // 2048 * 1024, T // 1024 * 1024):
        n = min(1024, T - i)
        assert torch.equal(r.y[i:i + n], few.y[:n]) and torch.equal(r.q.scales[i:i + n], few.q.scales[:n])
        assert torch.equal(r.q.codes[i:i + n].view(torch.uint8), few.q.codes[:n].view(torch.uint8))
    del r, few
    dx, dg = Q.add_rmsnorm_backward(x, x, g, need_dgamma=False)
    few = Q.add_rmsnorm_backward(part, part, g, need_dgamma=False)[0]
    assert dg is None and torch.equal(dx[T // 1024 * 1024:], few[:T - T // 1024 * 1024])


FIRST = """
import torch, quantile_balanced_routing_gb300 as Q
Q.route_qb(torch.randn(4, 32, device="cuda"), 2)        # the library's first call, before any capture
u8 = lambda *s: torch.randint(100, 120, s, dtype=torch.uint8, device="cuda")
gate, up, out = Q.Mxfp4(u8(8, 64, 128), u8(8, 64, 8)), Q.Mxfp4(u8(8, 64, 128), u8(8, 64, 8)), Q.Mxfp4(u8(8, 256, 32), u8(8, 256, 2))
wide, deep = Q.Mxfp4(u8(8192, 512), u8(8192, 32)), Q.Mxfp4(u8(16, 4128), u8(16, 258))
big = [Q.Mxfp4(u8(8, 1024, 512), u8(8, 1024, 32)) for _ in range(3)]
x, rows = torch.randn(64, 256, device="cuda").bfloat16(), torch.randn(64, 1024, device="cuda").bfloat16()
far, odd, long = torch.randn(3, 8256, device="cuda").bfloat16(), torch.randn(5, 33, device="cuda"), torch.randn(4000, 1024, device="cuda").bfloat16()
idx = torch.randint(0, 8, (64, 4), device="cuda").int()
w, ones = torch.rand(64, 4, device="cuda"), torch.ones(8192, device="cuda")
def run():
    n, m = Q.add_rmsnorm(x, ones[:256], mxfp8=True), Q.add_rmsnorm(long, ones[:1024], residual=long, mxfp8=True)
    return [n.y, n.q.scales, m.y, Q.add_rmsnorm(odd, ones[:33]).y, *Q.add_rmsnorm_backward(odd, odd, ones[:33]),
            *Q.add_rmsnorm_backward(long, long, ones[:1024]), *Q.add_rmsnorm_backward(x, x, ones[:256]),
            Q.mxfp4_matvec(rows, wide), Q.mxfp4_matvec(far, deep), Q.mxfp4_experts(x, idx, w, gate, up, out),
            Q.mxfp4_experts(n.q, idx, w, gate, up, out, gamma=ones[:256]), Q.mxfp4_experts(rows, idx, w, *big)]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, run()))
assert Q.qbmoe_status(None, None) == 0
print("as later")
"""


def test_captured_before_any_other_call_of_theirs():
    p = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "as later" in p.stdout, p.stderr[-3000:]


def test_two_host_threads_at_once():
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(3)
    made = [[weights(r, 6, 96, 160)[0], weights(r, 6, 96, 160)[0], weights(r, 6, 160, 96)[0]] for _ in range(2)]
    big = [weights(r, 904, 1024)[0] for _ in range(2)]
    rows = [torch.randn(700, 1024, device="cuda").bfloat16() for _ in range(2)]
    x = [torch.randn(9, 160, device="cuda").bfloat16() for _ in range(2)]
    idx, w = torch.from_numpy(r.randint(0, 6, (9, 3)).astype(np.int32)).cuda(), torch.rand(9, 3, device="cuda")
    g = torch.ones(1024, device="cuda")

    def run(i):
        return Q.mxfp4_experts(x[i], idx, w, *made[i]), Q.mxfp4_matvec(rows[i], big[i]), Q.add_rmsnorm(rows[i], g, mxfp8=True).y, \
            *Q.add_rmsnorm_backward(rows[i], rows[i], g)

    want = [run(0), run(1)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()

    def many(i):
        with torch.cuda.stream(streams[i]):
            got = [run(i) for _ in range(30)]
        streams[i].synchronize()
        return all(torch.equal(a, b) for one in got for a, b in zip(one, want[i]))

    with ThreadPoolExecutor(max_workers=2) as pool:
        assert all(pool.map(many, range(2)))
