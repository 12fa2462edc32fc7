"""Attention of shared beginnings where one position takes nearly everything: what many small probabilities leave, held to the decode call's own bound."""
import pytest

from attention_common import check
from test_gpu_attention_prefix import Batch

pytestmark = pytest.mark.gpu


def peaked(kind, cache, dim, heads, members, shared, gap, at):
    """Scores of 0 but for shared position `at`, which has `gap` and whose values are 0 in every other element; all other values are 1."""
    b = Batch(kind, cache, "heads", dim, 64, heads, 1, members, shared, 60)
    one = 0x38 if cache == "e4m3" else 1.0
    b.c.planes[0].fill_(0), b.c.planes[1].fill_(one)
    for scale in b.c.scales:
        if scale is not None:
            scale.fill_(127)
    b.c.k[:], b.c.v[:] = 0.0, 1.0
    for row in b.first[:-1]:
        page, slot = int(b.table[row, at // 64]), at % 64
        b.c.planes[0][page, :, slot] = one
        b.c.planes[1][page, :, slot, ::2] = 0
        b.c.k[page, :, slot], b.c.v[page, :, slot, ::2] = 1.0, 0.0
    b.q.fill_(gap / dim ** 0.5)  # a score is dim of these, times dim ** -0.5
    return b


@pytest.mark.parametrize("kind,cache,dim,heads", [("f16", "f16", 32, 32), ("f16", "e4m3", 32, 16), ("f16", "e4m3", 160, 8), ("bf16", "bf16", 32, 32), ("f16", "f16", 128, 2)])
@pytest.mark.parametrize("gap,at", [(30.0, 3), (30.0, 9800), (21.5, 3)])
def test_peaked(kind, cache, dim, heads, gap, at):
    """Long runs of keys of one workgroup (20 tiles and more), which count nothing beside one of them."""
    b = peaked(kind, cache, dim, heads, [2], [39936], gap, at)
    for sharing in (False, True):
        out, lse = b.run(sharing=sharing)
        check(b.c, kind, b.q, out, lse, b.table, b.lengths)


@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("f16", "e4m3"), ("bf16", "bf16")])
@pytest.mark.parametrize("step", [0.2, 0.6, 0.9, 1.5, 7.0])
def test_rising_scores(kind, cache, step):
    """Scores that rise from tile to tile, by less and by more than the running maximum follows at once."""
    b = Batch(kind, cache, "heads", 64, 64, 1, 2, [3], [1280], 50, seed=3)
    one = 0x38 if cache == "e4m3" else 1.0
    # element e of a key of page 2 p + (e > 0) is 1 for e < p: a score is their number, in steps of `step`
    b.c.planes[0].fill_(0), b.c.k.fill(0.0)
    if b.c.scales[0] is not None:
        b.c.scales[0].fill_(127)
    for p in range(20):
        page = int(b.table[0, p])
        b.c.planes[0][page, 0, :, :p], b.c.k[page, 0, :, :p] = one, 1.0
    b.q.fill_(step * 64 ** 0.5)
    out, lse = b.run()
    check(b.c, kind, b.q, out, lse, b.table, b.lengths)
