"""Packed batches of very many sequences."""
import numpy as np
import pytest

import mx_reference as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,S", [(3000, 70000), (70001, 70000)])
def test_more_than_65535_sequences(T, S):
    """A share is within 2^-17 of the largest one (fp32 sums of at most T shares), a loss within twice that."""
    import quantile_balanced_routing_gb300 as Q
    r = np.random.RandomState(T)
    n, k = 8, 2
    x = torch.from_numpy(r.standard_normal((T, n)).astype(np.float32))
    idx = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :k].to(torch.int32).contiguous()
    off = np.concatenate([[0], np.sort(r.randint(0, T + 1, S - 1)), [T]]).astype(np.int32)
    got = Q.balance_loss(x.cuda(), idx.cuda(), torch.from_numpy(off).cuda())
    # the sequences that have tokens, by themselves
    some = np.flatnonzero(off[1:] > off[:-1])
    loss, counts, probs, tokens = M.balance(x.double().numpy(), idx.numpy(), np.append(off[some], T))
    full = lambda v: np.concatenate([v, np.zeros((1, *v.shape[1:]))])  # noqa: E731
    at = np.full(S, len(some))
    at[some] = np.arange(len(some))
    assert np.array_equal(got.counts.cpu().numpy(), full(counts)[at])
    assert np.array_equal(got.tokens.cpu().numpy(), full(tokens)[at])
    assert np.abs(got.probs.double().cpu().numpy() - full(probs)[at]).max() < 2.0 ** -17
    assert np.abs(got.loss.double().cpu().numpy() - full(loss)[at]).max() < 2.0 ** -16 * loss.max()
    dw, dl = r.standard_normal((T, k)).astype(np.float32), r.standard_normal(S).astype(np.float32)
    g = Q.router_backward(x.cuda(), idx.cuda(), dw=torch.from_numpy(dw).cuda(), dloss=torch.from_numpy(dl).cuda(),
                          counts=got.counts, tokens=got.tokens, seq_offsets=torch.from_numpy(off).cuda())
    want = M.router_grad(x.double().numpy(), idx.numpy(), dw, dl[some], counts, tokens, np.append(off[some], T))
    size = np.abs(dw).max() + (np.abs(dl[some]) * n / (k * tokens ** 2.0) * counts.max(1)).max()
    assert np.abs(g.double().cpu().numpy() - want).max() < 2.0 ** -17 * size
