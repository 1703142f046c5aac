"""Softcaps, epsilons and sizes at which the few-row calls and the norm stop taking arguments, on the host (no GPU needed)."""
import pytest

import quantile_balanced_routing_gb300 as Q

torch = pytest.importorskip("torch")

FAKE, BIG, INF = 1 << 20, 1 << 40, float("inf")   # aligned fake device address: never dereferenced by the host checks


@pytest.fixture(scope="module")
def lib():
    return Q.load_library()


@pytest.mark.parametrize("beta1,beta2,eps", [(INF, 25.0, 1e-6), (4.0, INF, 1e-6), (1e20, 1e20, 1e-6), (2.0 ** 64, 2.0 ** 63.5, 1e-6),
                                             (4.0, 25.0, INF), (1e39, 25.0, 1e-6), (4.0, 25.0, 1e39)])
def test_experts_refuses_infinite_softcaps_and_activations(lib, beta1, beta2, eps):
    """An infinite softcap makes every activation NaN (infinity times 0), and softcaps whose product passes fp32 infinite
    ones; an infinite epsilon makes every output zero."""
    assert lib.moe_mxfp4_experts(4, 2, 8, 64, 96, 3, FAKE, 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, beta1, beta2,
                                 FAKE, eps, FAKE, 64, FAKE, BIG, None) == Q.QBMOE_EINVAL


def test_python_names_what_is_wrong_with_softcaps_and_epsilons():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    gate, out = Q.Mxfp4(u8(3, 96, 32), u8(3, 96, 2)), Q.Mxfp4(u8(3, 64, 48), u8(3, 64, 3))
    x8 = Q.Mxfp8(u8(4, 64), u8(4, 2))
    args = [x8, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), gate, gate, out]
    for kw in (dict(beta1=1e20, beta2=1e20), dict(beta1=1e39), dict(beta2=1e-50), dict(eps=1e39)):
        with pytest.raises(Q.QbmoeError, match="beta1 beta2 is at most") as e:
            Q.mxfp4_experts(*args, **kw)
        assert e.value.code == Q.QBMOE_EINVAL
