"""Parts of larger MXFP4 tensors and offsets, which start where they start, give what copies of them give."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def quantised(*shape, seed):
    import quantile_balanced_routing_gb300 as Q
    g = torch.Generator(device="cuda").manual_seed(seed)
    return Q.mxfp4_quantize(torch.randn(*shape, generator=g, device="cuda"))


def part(q, cut):
    """(the slice, a copy of it)"""
    import quantile_balanced_routing_gb300 as Q
    return Q.Mxfp4(q.codes[cut], q.scales[cut]), Q.Mxfp4(q.codes[cut].clone(), q.scales[cut].clone())


def both(x, w, offsets, dy):
    import quantile_balanced_routing_gb300 as Q
    out = (Q.mxfp4_matmul(x, w, offsets), *Q.mxfp4_matmul_backward(dy, x, w, offsets))
    assert Q.qbmoe_status(None, None) == 0
    return out


@pytest.mark.parametrize("K", [32, 96, 512])
@pytest.mark.parametrize("first", [1, 2, 5])
def test_rows_from_any_row_on(K, first):
    x, xc = part(quantised(70, K, seed=K), slice(first, None))
    w = quantised(40, K, seed=1)
    dy = torch.randn(70 - first, 40, device="cuda").bfloat16()
    for got, want in zip(both(x, w, None, dy), both(xc, w, None, dy)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("K", [32, 96, 512])
def test_one_expert_of_many(K):
    w, wc = part(quantised(5, 8, K, seed=K), 3)
    x = quantised(20, K, seed=2)
    dy = torch.randn(20, 8, device="cuda").bfloat16()
    for got, want in zip(both(x, w, None, dy), both(x, wc, None, dy)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("start", [1, 2, 3])
def test_offsets_inside_a_larger_tensor(start):
    table = torch.zeros(12, dtype=torch.int32, device="cuda")
    table[start:start + 4] = torch.tensor([0, 7, 7, 30], device="cuda")
    x, w = quantised(30, 64, seed=3), quantised(3, 16, 64, seed=4)
    dy = torch.randn(30, 16, device="cuda").bfloat16()
    off = table[start:start + 4]
    for got, want in zip(both(x, w, off, dy), both(x, w, off.clone(), dy)):
        assert torch.equal(got, want)
