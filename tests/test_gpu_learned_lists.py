"""The example that runs the softmax-over-codes operators together."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_learned_lists():
    spec = importlib.util.spec_from_file_location(
        "learned_lists", os.path.join(ROOT, "examples", "learned_lists.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    n, k = 6000, 64
    out = example.main(n, k, 20)
    # untrained, every code is as probable as any other; training lowers the loss
    assert abs(out["losses"][0] - math.log(k)) < 1e-4
    assert out["losses"][-1] < 0.8 * out["losses"][0]
    # every row is in one list or two, and the lists are whole
    assert n <= out["entries"] <= 2 * n
    assert out["offsets"].shape == (k + 1,) and int(out["offsets"][-1]) == out["entries"]
    assert torch.equal(torch.unique(out["rows"]), torch.arange(n, dtype=torch.int32))
    assert out["visit"].shape == (4, 4) and bool((out["visit"] >= 0).all())
    assert bool(torch.isfinite(out["d_refined"]).all())
