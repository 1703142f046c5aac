"""Status and test hooks of the calls that take no context, from two host threads and streams."""
from concurrent.futures import ThreadPoolExecutor

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture
def other():
    """Runs a function in a second thread, always the same one."""
    with ThreadPoolExecutor(max_workers=1) as pool:
        yield lambda f: pool.submit(f).result()


@pytest.fixture
def product():
    import quantile_balanced_routing_gb300 as Q
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = (Q.mxfp4_quantize(torch.randn(r, 256, generator=g, device="cuda")) for r in (40, 128))
    torch.cuda.synchronize()
    return lambda: Q.mxfp4_matmul(x, w)


@pytest.fixture
def hooks():
    """Sets (wait limit, stall) of the calling thread; this thread's are put back afterwards."""
    import quantile_balanced_routing_gb300 as Q
    lib = Q.load_library()

    def arm(limit, stall):
        assert lib.qbmoe_set_wait_limit(None, limit) == 0 and lib.qbmoe_debug_stall(None, stall) == 0
    yield arm
    arm(0, 0)


def test_one_thread_does_not_take_the_timeout_of_another(other, product, hooks):
    import quantile_balanced_routing_gb300 as Q
    ask = lambda: Q.qbmoe_status(None, None)  # noqa: E731
    product()
    ask(), other(ask)                    # what earlier tests left
    hooks(200, 1)
    product()
    hooks(0, 0)
    torch.cuda.synchronize()
    assert other(ask) == Q.QBMOE_ETIMEOUT
    assert ask() == Q.QBMOE_ETIMEOUT
    assert ask() == 0 and other(ask) == 0


def test_hooks_are_those_of_the_thread_that_sets_them(other, product, hooks):
    import quantile_balanced_routing_gb300 as Q
    ask = lambda: Q.qbmoe_status(None, None)  # noqa: E731
    want = product()
    ask(), other(ask)
    hooks(200, 1)
    got = other(product)
    assert ask() == 0 and other(ask) == 0
    assert torch.equal(got, want)


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


def test_a_closed_layer_has_no_part_in_it(product, hooks):
    import quantile_balanced_routing_gb300 as Q
    lay = Q.LatentMoE(512, 512, 16, 2, 512, 0, max_tokens=32)
    lay.close()
    product()
    Q.qbmoe_status(None, None)
    hooks(200, 1)
    product()
    hooks(0, 0)
    assert lay.status() == 0
    assert Q.qbmoe_status(None, None) == Q.QBMOE_ETIMEOUT
