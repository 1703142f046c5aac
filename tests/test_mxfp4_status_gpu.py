"""Status of the calls that take no context."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture
def product():
    import quantile_balanced_routing_gb300 as Q
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = (Q.mxfp4_quantize(torch.randn(r, 256, generator=g, device="cuda")) for r in (40, 128))
    torch.cuda.synchronize()
    return lambda: Q.mxfp4_matmul(x, w)


def test_status_of_a_stream_does_not_wait_for_others(product):
    """A quarter of a second's work on the default stream is still running when another stream's status comes back."""
    import quantile_balanced_routing_gb300 as Q
    s = torch.cuda.Stream()
    product()
    Q.qbmoe_status(None, None)
    with torch.cuda.stream(s):
        product()
    done = torch.cuda.Event()
    torch.cuda._sleep(500_000_000)
    done.record()
    assert Q.qbmoe_status(None, s.cuda_stream) == 0
    assert not done.query()
    torch.cuda.synchronize()
