"""Attention of shared beginnings with scales of every sign, over whole and partial tiles of what is shared and with missing pages."""
import pytest
import torch

from attention_common import check
from cache_common import fmt_of
from gpu_common import dev, require_gpu
from test_gpu_attention_prefix import FAR, Batch

pytestmark = pytest.mark.gpu


def run(b, scale, softcap=0.0, sharing=True):
    api = require_gpu()
    n, hq, _ = b.q.shape
    out, lse = torch.full_like(b.q, float("nan")), torch.full((n, hq), 99.0, device="cuda")
    ws = torch.zeros(api.mxattn_prefix_workspace_size(b.c.c, n, hq, len(b.shared), FAR, FAR), dtype=torch.uint8, device="cuda")
    api.mxattn_prefix_run(b.c.c, fmt_of(api, b.kind), b.q, out, dev(b.table), dev(b.lengths), FAR, dev(b.first), dev(b.shared), FAR, scale, lse=lse,
                          softcap=softcap, workspace=ws if sharing else None)
    return out, lse


@pytest.mark.parametrize("kind,cache,dim", [("f16", "f16", 128), ("bf16", "bf16", 64), ("f16", "e4m3", 64), ("bf16", "e4m3", 128), ("f16", "f16", 256), ("bf16", "e4m3", 256)])
@pytest.mark.parametrize("scale", [0.0, -0.0, -0.11, 1e-30])
@pytest.mark.parametrize("missing", [False, True])
def test_scales(kind, cache, dim, scale, missing):
    """A scale of 0 gives the mean of the values, a negative one turns the scores: behind 64 and 192 positions, half a tile of 128 at the end, and behind 256."""
    b = Batch(kind, cache, "heads", dim, 16, 2, 4, [3, 2, 2], [192, 64, 256], 40)
    if missing:
        b.table[:3, [1, 5, 6, 7, 8, 11]] = -1  # all of a run of 64 but its last page among them
        b.table[5:7, :16] = -1
    out, lse = run(b, scale)
    check(b.c, kind, b.q, out, lse, b.table, b.lengths, scale=scale)


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_scales_with_a_cap(cache, scale):
    b = Batch("f16", cache, "slots", 128, 32, 2, 6, [5], [320], 50)
    b.table[:, 2] = -1
    out, lse = run(b, scale, softcap=2.0)
    check(b.c, "f16", b.q, out, lse, b.table, b.lengths, softcap=2.0, scale=scale)


def test_infinite_score_times_zero():
    """A score that is infinite is NaN with a scale of 0, with and without sharing."""
    b = Batch("f16", "f16", "heads", 128, 16, 2, 4, [3], [192], 20)
    b.c.planes[0][int(b.table[0, 3]), 1, 2, 9] = float("inf")
    (out, lse), (want, want_lse) = run(b, 0.0), run(b, 0.0, sharing=False)
    assert bool(want[:, 4:].isnan().all()) and not bool(want[:, :4].isnan().any())
    assert torch.equal(out.isnan(), want.isnan()) and torch.equal(lse.isnan(), want_lse.isnan())
