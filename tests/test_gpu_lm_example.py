"""The post-training example runs all the losses together and trains: the distillation,
preference and balance losses go down (the policy's own value is the mean advantage
on-policy and only its KL term shows)."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_routed_lm_example_trains():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sinkhorn_point_cloud_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import routed_lm_step
    h = routed_lm_step.train(steps=30, report=False)
    first, last = h[0], h[-1]
    assert last["distil"] < first["distil"], (first, last)
    assert abs(first["prefer"] - 0.6931) < 1e-3 and last["prefer"] < 0.5 * first["prefer"], (first, last)
    assert last["margin"] > 1.0
    assert last["balance"] < first["balance"], (first, last)
    assert abs(first["kl"]) < 1e-6 and last["kl"] > 0
