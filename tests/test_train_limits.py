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
