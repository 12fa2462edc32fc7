"""The example's attention layer: int8 weights, rotation, append, attention, forks and compaction together."""
import importlib.util
import os

import pytest

from gpu_common import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,bound", [("fp16", 0.01), ("e4m3", 0.2)])
def test_decode_step(kind, bound):
    """Outputs stay near fp32's. A step's output is a sum of 512 products of attention outputs (below 1 in size,
    off by fp16 steps of 2^-11, or E4M3's of 2^-4 that averaging over keys reduces) with weights of size
    512^-1/2: a few 2^-11, or some 2^-4."""
    require_gpu()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    say(f"decode step over a {kind} cache")
    worst = m.main(kind, 24)
    say(f"largest difference {worst:.5f}")
    assert 0.0 < worst <= bound
