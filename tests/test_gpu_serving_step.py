"""The serving example: tables on the device, norm, products of 8-bit integers, append, attention behind a shared prompt together,
eager and as a replayed graph."""
import importlib.util
import os

import pytest
import torch

from gpu_common import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,bound", [("fp16", 0.12), ("e4m3", 0.3)])
def test_serving_step(kind, bound):
    """Outputs stay near fp32's. A normalised row's largest element is about 4, so its 8-bit integers are off by 2^-6 at most and
    2^-6 / sqrt(3) in the mean; sums of 512 such errors with weights of size 512^-1/2 put that on q, k and v, of size 1; scores, of 64
    products scaled by 1 / 8, are off by about 2 * 2^-6 / sqrt(3) = 0.018, and outputs, means of values, by that part of their size and the
    values' own 0.009: 0.02, of which the largest of some 10^5 is five times that at most (E4M3 keys and values: 2^-4 / sqrt(3) = 0.036 more, which the mean over keys reduces,
    and scores off by that: 0.06). A wrong row, page or position puts them off by about 1."""
    require_gpu()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serving_step.py")
    spec = importlib.util.spec_from_file_location("serving_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    say(f"serving step over a {kind} cache")
    worst, last = m.main(kind, 40)
    say(f"largest difference {worst:.5f}; as a graph")
    assert 0.0 < worst <= bound
    again, replayed = m.main(kind, 40, graph=True)
    say(f"largest difference {again:.5f}")
    assert again == worst and torch.equal(last, replayed)
