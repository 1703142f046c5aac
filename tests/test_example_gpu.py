"""The quantisation-aware training example learns."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_qat_example_learns():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import qat_experts
    finally:
        sys.path.pop(0)
    h = qat_experts.train(steps=60, log=None)
    first, last = (sum(t for t, _ in part) / len(part) for part in (h[:10], h[-10:]))
    assert last < 0.8 * first
    assert all(a > 0.9 for _, a in h)       # about 1 when balanced
