"""Page copies over layers, bit for bit, and the host pool driving them."""
import numpy as np
import pytest
import torch

from cache_common import Cache
from gpu_common import dev, require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("order", ["heads", "slots"])
@pytest.mark.parametrize("layers,pages,page,heads,dim,n", [(1, 2, 1, 1, 32, 1), (3, 40, 5, 3, 96, 17), (33, 6, 16, 2, 64, 3),
                                                           (2, 300, 24, 8, 128, 150), (2, 9, 256, 12, 256, 4)])
def test_copy_pages(kind, order, layers, pages, page, heads, dim, n):
    api = require_gpu()
    say(f"copy {kind} {order} layers={layers} pages={pages} page={page} heads={heads} dim={dim} pairs={n}")
    caches = [Cache(kind, order, pages, page, heads, dim, 10 + i, paired=kind != "e4m3" and layers == 3) for i in range(layers)]
    before = [[t.cpu().clone() for t in c.planes + [s for s in c.scales if s is not None]] for c in caches]
    pairs = np.random.Generator(np.random.PCG64(n)).permutation(pages)[:2 * n].reshape(n, 2).astype(np.int32)
    bad = np.array([[0, pages], [-1, 1], [1, 1], [pages + 5, 0], [2 ** 31 - 1, 0], [0, -2 ** 31]], np.int32)
    api.mxkv_copy_run([c.c for c in caches], dev(np.concatenate([bad[:3], pairs, bad[3:]])))
    torch.cuda.synchronize()
    for c, was in zip(caches, before):
        for got, w in zip(c.planes + [s for s in c.scales if s is not None], was):
            w[pairs[:, 1]] = w[pairs[:, 0]]
            assert torch.equal(got.cpu().contiguous().view(torch.uint8), w.contiguous().view(torch.uint8))


def test_copy_nothing():
    api = require_gpu()
    c = Cache("f16", "heads", 2, 4, 1, 8, 1)
    api.mxkv_copy_run([c.c], torch.zeros((0, 2), dtype=torch.int32, device="cuda"))
    api.mxkv_copy_run([], torch.zeros((3, 2), dtype=torch.int32, device="cuda"))


def test_pool_moves_keep_every_sequence():
    """Sequences written, forked, grown, freed and compacted through the pool read back what was written."""
    api = require_gpu()
    say("pool: grow, fork, free, compact")
    page, heads, dim, seqs, cols = 4, 2, 32, 5, 6
    c = Cache("f16", "slots", 20, page, heads, dim, 3)
    pool, text, rng = api.KVPool(20, page, seqs, cols), [[] for _ in range(seqs)], np.random.Generator(np.random.PCG64(8))

    def move(pairs):
        if pairs:
            api.mxkv_copy_run([c.c], dev(np.array(pairs, np.int32)))

    def grow(s, n):
        at = len(text[s])
        move(pool.resize(s, at + n))
        new = rng.integers(0, 1000, n)
        kv = torch.from_numpy(np.broadcast_to(new[:, None, None], (n, heads, dim)).astype(np.float16)).cuda()
        api.mxkv_append_run(c.c, api.MX_F16, kv, kv, dev(np.arange(at, at + n, dtype=np.int32)), dev(pool.table()),
                            seq=dev(np.full(n, s, np.int32)))
        text[s] += list(new)

    def check():
        for s in range(seqs):
            j = np.arange(len(text[s]))
            at = pool.table()[s][j // page]
            assert np.array_equal(c.planes[0].cpu().numpy()[at, j % page, 1, 5], np.array(text[s], np.float16))

    grow(0, 10)
    pool.fork(0, 1)
    pool.fork(0, 2)
    text[1], text[2] = list(text[0]), list(text[0])
    for s in (0, 1, 2):
        grow(s, 3)
    check()
    pool.resize(0, 0)
    text[0] = []
    grow(3, 9)
    pool.reorder([1, 1, 2, 3, 0])
    text = [list(text[i]) for i in (1, 1, 2, 3, 0)]
    grow(0, 1)
    check()
    pool.resize(2, 3)
    text[2] = text[2][:3]
    move(pool.compact())
    assert pool.table().max() == pool.used - 1
    check()
    grow(2, 7)
    check()
    pool.close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_copy_pairs_of_several_launches(kind):
    """A list of pairs, most of them ignored, whose words pass 2^31: valid ones at its ends and at the launches' borders."""
    api = require_gpu()
    page, heads, dim = 256, 8, 128
    words = page * heads * dim * (1 if kind == "e4m3" else 2) // 16
    most = (2 ** 31 - 256) // words
    n = 2 * most + 5
    say(f"copy {kind}: {n} pairs of {words} words")
    c = Cache(kind, "heads", 12, page, heads, dim, 3)
    planes = c.planes + [s for s in c.scales if s is not None]
    before = [t.cpu().clone() for t in planes]
    pairs = np.full((n, 2), -1, np.int32)
    real = {0: (0, 6), most - 1: (1, 7), most: (2, 8), 2 * most - 1: (3, 9), 2 * most: (4, 10), n - 1: (5, 11)}
    for i, p in real.items():
        pairs[i] = p
    api.mxkv_copy_run([c.c], dev(pairs))
    torch.cuda.synchronize()
    for got, w in zip(planes, before):
        w[6:] = w[:6]
        assert torch.equal(got.cpu().view(torch.uint8), w.view(torch.uint8))
