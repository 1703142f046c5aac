"""moe_balance_loss and moe_router_backward against their formulas in 64 bits
and against differences.

Tolerances.  A score from the hardware exponential is within about
|x| 2^-24 + 2^-21 of its value, a sum of n <= 1024 fp32 terms within 2^-19 of
the sum of magnitudes (a lane's 32 terms, then 5 levels): 2^-17 of the largest
magnitude covers shares, losses and gradients at |x| <= 30, and 2^-14 at
|x| <= 80; bf16 outputs add 2^-8 of their own value.
"""
import numpy as np
import pytest

import mx_reference as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CASES = [
    # T, n, k, sequences, padding, dtype, kind
    (1, 2, 1, 1, 0.0, "float32", "normal"),
    (1, 1024, 32, 1, 0.0, "bfloat16", "normal"),
    (64, 32, 4, 1, 0.0, "float32", "normal"),
    (257, 101, 7, 3, 0.2, "bfloat16", "normal"),       # odd rows: element-wise loads
    (300, 99, 5, 4, 0.2, "float32", "normal"),
    (1000, 896, 16, 9, 0.5, "float32", "normal"),
    (77, 40, 40 - 8, 77, 0.0, "float32", "normal"),    # a sequence per token
    (50, 24, 3, 200, 0.3, "bfloat16", "normal"),       # more sequences than tokens
    (700, 256, 8, 5, 1.0, "float32", "normal"),        # padding only
    (130, 64, 6, 2, 0.1, "float32", "extreme"),        # infinities, the clamp, equal rows
    (5000, 72, 4, 3, 0.1, "bfloat16", "normal"),
]


def case(T, n, k, S, pad, dtype, kind, seed=0):
    r = np.random.RandomState(seed + 31 * T + n)
    x = (r.standard_normal((T, n)) + r.standard_normal(n)).astype(np.float32)
    if kind == "extreme":
        x[0::7] *= 40.0
        x[1::7] = -np.inf
        x[2::7, ::2] = np.inf
        x[3::7] = 0.0
        x[4::7] = -100.0
    x = torch.from_numpy(x).to(getattr(torch, dtype))
    idx = torch.sort(x.float(), dim=1, descending=True, stable=True)[1][:, :k].to(torch.int32).contiguous()
    off = np.concatenate([[0], np.sort(r.randint(0, T + 1, S - 1)), [T]]).astype(np.int32)
    mask = r.random_sample(T) >= pad
    dw = r.standard_normal((T, k)).astype(np.float32)
    dl = r.standard_normal(S).astype(np.float32)
    return x, idx, off, mask, dw, dl


def near(got, want, size, rel, own=0.0):
    got = got.double().cpu().numpy() if hasattr(got, "cpu") else got
    assert got.shape == want.shape
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > rel * size + own * np.abs(want)
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - want).max(), size)


@pytest.mark.parametrize("T,n,k,S,pad,dtype,kind", CASES)
def test_loss_counts_and_shares(T, n, k, S, pad, dtype, kind):
    import quantile_balanced_routing_gb300 as Q
    x, idx, off, mask, _, _ = case(T, n, k, S, pad, dtype, kind)
    r = Q.balance_loss(x.cuda(), idx.cuda(), seq_offsets=torch.from_numpy(off).cuda(),
                       token_mask=torch.from_numpy(mask).cuda())
    loss, counts, probs, tokens = M.balance(x.double().numpy(), idx.numpy(), off, mask)
    assert np.array_equal(r.counts.cpu().numpy(), counts)
    assert np.array_equal(r.tokens.cpu().numpy(), tokens)
    rel = 2.0 ** (-17 if kind == "normal" else -14)
    near(r.probs, probs, max(probs.max(), 1e-30), rel)
    near(r.loss, loss, np.maximum(loss, 1e-30), 2 * rel)


@pytest.mark.parametrize("parts", ["both", "weights", "loss"])
@pytest.mark.parametrize("T,n,k,S,pad,dtype,kind", CASES)
def test_router_gradient(T, n, k, S, pad, dtype, kind, parts):
    import quantile_balanced_routing_gb300 as Q
    x, idx, off, mask, dw, dl = case(T, n, k, S, pad, dtype, kind)
    dw, dl = None if parts == "loss" else dw, None if parts == "weights" else dl
    _, counts, _, tokens = M.balance(x.double().numpy(), idx.numpy(), off, mask)
    c, t = torch.from_numpy(counts.astype(np.int32)).cuda(), torch.from_numpy(tokens.astype(np.int32)).cuda()
    up = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    g = Q.router_backward(x.cuda(), idx.cuda(), dw=up(dw), dloss=up(dl), counts=c if dl is not None else None,
                          tokens=t if dl is not None else None, seq_offsets=up(off), token_mask=up(mask))
    assert g.dtype == x.dtype
    want = M.router_grad(x.double().numpy(), idx.numpy(), dw, dl, counts, tokens, off, mask)
    # the terms subtract from sums of their own size: one row's largest magnitudes
    size = 0.0
    if dw is not None:
        size = size + np.abs(dw).max()
    if dl is not None:
        f = np.abs(dl) * n / (k * np.maximum(1, tokens) ** 2.0) * counts.max(1)
        size = size + f.max()
    near(g, want, size, 2.0 ** (-17 if kind == "normal" else -14), 2.0 ** -8 if dtype == "bfloat16" else 0.0)
    assert not g[~torch.from_numpy(mask).cuda()].any()


def test_gradient_against_differences():
    """Central differences of the 64-bit objective, h = 1e-4: their own error is
    about h^2 = 1e-8 of the third derivative, far below 2^-17 of the largest term."""
    import quantile_balanced_routing_gb300 as Q
    x, idx, off, mask, dw, dl = case(40, 24, 5, 3, 0.2, "float32", "normal")
    r = Q.balance_loss(x.cuda(), idx.cuda(), seq_offsets=torch.from_numpy(off).cuda(),
                       token_mask=torch.from_numpy(mask).cuda())
    g = Q.router_backward(x.cuda(), idx.cuda(), dw=torch.from_numpy(dw).cuda(), dloss=torch.from_numpy(dl).cuda(),
                          counts=r.counts, tokens=r.tokens, seq_offsets=torch.from_numpy(off).cuda(),
                          token_mask=torch.from_numpy(mask).cuda()).cpu().numpy()
    counts, tokens = r.counts.cpu().numpy(), r.tokens.cpu().numpy()
    xs = x.double().numpy()
    h = 1e-4
    for t, j in [(0, 0), (3, idx[3, 0]), (17, idx[17, 4]), (22, 23), (39, 5), (39, idx[39, 2])]:
        up, dn = xs.copy(), xs.copy()
        up[t, j] += h
        dn[t, j] -= h
        d = (M.objective(up, idx.numpy(), dw, dl, counts, tokens, off, mask) -
             M.objective(dn, idx.numpy(), dw, dl, counts, tokens, off, mask)) / (2 * h)
        assert abs(g[t, j] - d) < 2.0 ** -17 * (np.abs(dw).max() + np.abs(dl).max() * 24) + 1e-6


def test_balanced_batch_has_loss_one():
    """Every expert chosen equally often: the loss is n/(kT) * (kT/n) * sum of shares = 1."""
    import quantile_balanced_routing_gb300 as Q
    T, n, k = 96, 32, 4
    x = torch.randn(T, n, generator=torch.Generator().manual_seed(1)).cuda()
    idx = ((torch.arange(T)[:, None] * k + torch.arange(k)) % n).to(torch.int32).cuda()
    r = Q.balance_loss(x, idx)
    assert r.counts.min() == r.counts.max() == T * k // n
    assert abs(float(r.loss) - 1.0) < 2.0 ** -17


def test_nan_stays_in_its_place():
    """A NaN in padding is not read; in a valid token it shows in that sequence's loss and that token's gradient."""
    import quantile_balanced_routing_gb300 as Q
    x, idx, _, _, dw, _ = case(60, 32, 4, 1, 0.0, "float32", "normal")
    off = torch.tensor([0, 30, 60], dtype=torch.int32).cuda()
    mask = torch.ones(60, dtype=torch.bool)
    mask[10] = False
    x[10, 3] = float("nan")
    x[40, 7] = float("nan")
    r = Q.balance_loss(x.cuda(), idx.cuda(), seq_offsets=off, token_mask=mask.cuda())
    assert torch.isfinite(r.loss[0]) and torch.isnan(r.loss[1])
    g = Q.router_backward(x.cuda(), idx.cuda(), dw=torch.from_numpy(dw).cuda(), dloss=torch.ones(2).cuda(),
                          counts=r.counts, tokens=r.tokens, seq_offsets=off, token_mask=mask.cuda()).cpu()
    assert not g[10].any()
    assert torch.isnan(g[40]).any()
    assert torch.isfinite(torch.cat((g[:40], g[41:]))).all()


def test_strided_rows_absent_routes_and_in_place():
    import quantile_balanced_routing_gb300 as Q
    x, idx, _, _, dw, _ = case(65, 48, 6, 1, 0.0, "float32", "normal")
    idx[5, 2] = -1                                  # no route
    idx[6, :] = -1                                  # a token that went nowhere
    wide = torch.full((65, 61), float("nan"))
    for start in (0, 4, 5):                         # rows on and off 16-byte boundaries
        buf = wide.clone().cuda()
        buf[:, start:start + 48] = x.cuda()
        v = buf[:, start:start + 48]
        r = Q.balance_loss(v, idx.cuda())
        loss, counts, probs, tokens = M.balance(x.double().numpy(), idx.numpy())
        assert np.array_equal(r.counts.cpu().numpy(), counts)
        near(r.loss, loss, loss, 2.0 ** -16)
        want = M.router_grad(x.double().numpy(), idx.numpy(), dw, np.ones(1), counts, tokens)
        Q.router_backward(v, idx.cuda(), dw=torch.from_numpy(dw).cuda(), dloss=torch.ones(1).cuda(), counts=r.counts,
                          tokens=r.tokens, out=v)
        near(v, want, np.abs(dw).max() + 48.0 / 6 / 65, 2.0 ** -17)
        assert torch.isnan(buf[:, :start]).all() and torch.isnan(buf[:, start + 48:]).all()


def test_repeatable_and_on_another_stream():
    import quantile_balanced_routing_gb300 as Q
    x, idx, off, mask, dw, dl = (v if not isinstance(v, np.ndarray) else torch.from_numpy(v)
                                 for v in case(3000, 896, 16, 4, 0.1, "float32", "normal"))
    x, idx, off, mask, dw, dl = (v.cuda() for v in (x, idx, off, mask, dw, dl))

    def both(stream=None):
        r = Q.balance_loss(x, idx, seq_offsets=off, token_mask=mask, stream=stream)
        return r + (Q.router_backward(x, idx, dw=dw, dloss=dl, counts=r.counts, tokens=r.tokens, seq_offsets=off,
                                      token_mask=mask, stream=stream),)
    a = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = both(s)
    s.synchronize()
    for u, v in zip(a, b):
        assert torch.equal(u, v)
