"""The router's gradient where scores are tiny: tokens whose logits lie around the clamp at -80.

A score there is about 2^-115, its reciprocal 2^115: a product of the reciprocal with
a large upstream gradient, or of the score with a small one, leaves fp32's normal
range although the gradient itself does not.

Tolerance.  Weights and shares are quotients of scores within |x| 2^-24 + 2^-21 of their
values, |x| <= 80: 2^-16 covers a quotient and the rounding of the sums, and the two
differences that make a gradient (d - mean, f - D) are bounded by twice the largest
term: 2^-14 of the largest term.
"""
import numpy as np
import pytest

import mx_reference as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def saturated(T, n, k, lo, hi, seed):
    r = np.random.RandomState(seed)
    x = r.uniform(lo, hi, (T, n)).astype(np.float32)
    idx = np.argsort(-x, axis=1, kind="stable")[:, :k]
    idx[1::2] = np.argsort(x, axis=1, kind="stable")[1::2, :k]       # the lowest: where the clamp holds
    return r, torch.from_numpy(x), torch.from_numpy(np.ascontiguousarray(idx).astype(np.int32))


@pytest.mark.parametrize("n,k", [(16, 2), (101, 7), (896, 16)])      # 16-byte rows, odd rows, the layer's
@pytest.mark.parametrize("size", [2e4, 1e30, 1e-10, 1e-20])
@pytest.mark.parametrize("lo,hi", [(-85.0, -79.0), (-80.0, -70.0)])
def test_mixture_weights_of_tiny_scores(n, k, size, lo, hi):
    import quantile_balanced_routing_gb300 as Q
    r, x, idx = saturated(40, n, k, lo, hi, n)
    dw = (size * r.choice([-1.0, 0.5, 1.0], (40, k))).astype(np.float32)
    g = Q.router_backward(x.cuda(), idx.cuda(), dw=torch.from_numpy(dw).cuda()).double().cpu().numpy()
    want = M.router_grad(x.numpy(), idx.numpy(), dw, None, None, None)
    assert np.isfinite(g).all()
    assert (g[x.numpy() < -80] == 0).all()
    assert np.abs(g - want).max() < 2.0 ** -14 * np.abs(dw).max()


@pytest.mark.parametrize("n,k", [(16, 2), (101, 7), (896, 16)])
@pytest.mark.parametrize("size", [1e6, 1e-6, 1e-12])
def test_balance_loss_of_tiny_scores(n, k, size):
    import quantile_balanced_routing_gb300 as Q
    _, x, idx = saturated(40, n, k, -80.5, -76.0, n)
    r = Q.balance_loss(x.cuda(), idx.cuda())
    dl = np.array([size], np.float32)
    g = Q.router_backward(x.cuda(), idx.cuda(), dloss=torch.from_numpy(dl).cuda(), counts=r.counts, tokens=r.tokens)
    g, counts = g.double().cpu().numpy(), r.counts.cpu().numpy()
    want = M.router_grad(x.numpy(), idx.numpy(), None, dl, counts, r.tokens.cpu().numpy())
    f = size * n / (k * 40.0 ** 2) * counts.max()
    assert np.isfinite(g).all()
    assert (g[x.numpy() < -80] == 0).all()
    # a token's share of every expert is about 1 / n: so is the size of its gradients
    assert np.abs(g - want).max() < 2.0 ** -14 * f * (M.scores(x.numpy()) / M.scores(x.numpy()).sum(1, keepdims=True)).max()


@pytest.mark.parametrize("n", [32, 33])
def test_nan_of_an_expert_that_was_not_chosen(n):
    """Without a balance loss only the chosen scores enter a token's gradient: a NaN elsewhere stays in its place."""
    import quantile_balanced_routing_gb300 as Q
    r, x, idx = saturated(20, n, 3, -3.0, 3.0, n)
    dw = torch.from_numpy(r.standard_normal((20, 3)).astype(np.float32)).cuda()
    clean = Q.router_backward(x.cuda(), idx.cuda(), dw=dw)
    other = next(j for j in range(n) if j not in idx[7].tolist())
    x[7, other] = float("nan")
    g = Q.router_backward(x.cuda(), idx.cuda(), dw=dw)
    keep = torch.ones(20, n, dtype=torch.bool)
    keep[7, other] = False
    assert torch.equal(g.cpu()[keep], clean.cpu()[keep])


def one_token_sequences(T, n, k):
    x = torch.empty(T, n).uniform_(-80, 80, generator=torch.Generator().manual_seed(n))
    idx = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :k].to(torch.int32).contiguous()
    return x, idx, torch.arange(T + 1, dtype=torch.int32)


@pytest.mark.parametrize("n", [64, 63])
def test_scores_keep_fp32_over_the_whole_range(n):
    """Shares of single tokens, element by element.  A score is within 2^-21 of its value: 2^-22 for the exponential,
    2^-23 for the reciprocal, 2^-24 for each of two roundings.  Its sum adds 8 roundings, the quotient 3: 2^-19 covers
    a share.  (An exponent rounded once before the exponential is off by up to 115 2^-25, 2^-18 of the score.)"""
    import quantile_balanced_routing_gb300 as Q
    x, idx, off = one_token_sequences(512, n, 4)
    r = Q.balance_loss(x.cuda(), idx.cuda(), off.cuda())
    loss, _, want, _ = M.balance(x.double().numpy(), idx.numpy(), off.numpy())
    got = r.probs.double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -19 * want).all()
    assert (np.abs(r.loss.double().cpu().numpy() - loss) <= 2.0 ** -18 * loss).all()


@pytest.mark.parametrize("n", [64, 63])
def test_gradients_keep_fp32_over_the_whole_range(n):
    """Element by element, against the size of the terms that an element is the difference of: its slope over the sum
    of scores times the largest gradient.  Slope and quotient are within 2^-18.5, the mean within 2^-19.5: 2^-17."""
    import quantile_balanced_routing_gb300 as Q
    x, idx, off = one_token_sequences(512, n, 4)
    r = np.random.RandomState(n)
    dw, dl = r.standard_normal((512, 4)).astype(np.float32), r.standard_normal(512).astype(np.float32)
    xs, up = x.double().numpy(), lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    _, counts, _, tokens = M.balance(xs, idx.numpy(), off.numpy())
    s = M.scores(xs)
    slope = s * M.scores(-xs)
    chosen = np.zeros(s.shape)
    np.put_along_axis(chosen, idx.numpy(), 1.0, 1)
    g = Q.router_backward(x.cuda(), idx.cuda(), dw=up(dw)).double().cpu().numpy()
    want = M.router_grad(xs, idx.numpy(), dw, None, counts, tokens, off.numpy())
    size = slope / (s * chosen).sum(1, keepdims=True) * np.abs(dw).max(1, keepdims=True)
    assert (np.abs(g - want) <= 2.0 ** -17 * size * chosen).all()
    g = Q.router_backward(x.cuda(), idx.cuda(), dloss=up(dl), counts=up(counts.astype(np.int32)),
                          tokens=up(tokens.astype(np.int32)), seq_offsets=off.cuda()).double().cpu().numpy()
    want = M.router_grad(xs, idx.numpy(), None, dl, counts, tokens, off.numpy())
    size = slope / s.sum(1, keepdims=True) * (np.abs(dl) * n / 4)[:, None]
    assert (np.abs(g - want) <= 2.0 ** -17 * size).all()


@pytest.mark.parametrize("T,n,k", [(2048, 896, 16), (4000, 64, 6)])
def test_gradients_are_as_near_as_plain_fp32(T, n, k):
    """The error's norm against the formula is at most a quarter above that of its plain evaluation in 32-bit arithmetic
    (each share times its complement, p c (f - D) and w c (dw - mean)), which rounds as often."""
    import quantile_balanced_routing_gb300 as Q
    g = torch.Generator().manual_seed(n)
    new = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = new(T, n) + 1.4 * new(n)
    idx = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :k].to(torch.int32).contiguous()
    dw, dl = 0.1 * new(T, k), torch.tensor([0.01])
    r = Q.balance_loss(x.cuda(), idx.cuda())
    got = Q.router_backward(x.cuda(), idx.cuda(), dw=dw.cuda(), dloss=dl.cuda(), counts=r.counts, tokens=r.tokens)

    def formula(x, dw, f):
        s, c = 1 / (1 + torch.exp(-x)), 1 / (1 + torch.exp(x))
        p, i = s / s.sum(1, keepdim=True), idx.long()
        w = s.gather(1, i)
        w = w / w.sum(1, keepdim=True)
        return (p * c * (f - (f * p).sum(1, keepdim=True))).scatter_add(
            1, i, w * c.gather(1, i) * (dw - (dw * w).sum(1, keepdim=True)))
    counts = r.counts.cpu()
    want = formula(x.double(), dw.double(), counts.double() * (dl.double() * n / (k * T * T)))
    plain = formula(x, dw, counts.float() * (dl * n / (k * T * T)))
    assert float((got.cpu() - want).norm()) <= 1.25 * float((plain - want).norm())
