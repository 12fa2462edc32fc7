"""Attention of one new token over rows that are cut into shares: masks, missing pages, NaN in places that are not attended, every
head size and page size that has a kernel of its own, two tiles of query heads, and bounds far above the lengths."""
import numpy as np
import pytest
import torch

from attention_common import COUNTERS, attend, check, hide, workspace
from cache_common import Cache, f64, normal, tables
from gpu_common import require_gpu, say

pytestmark = pytest.mark.gpu


def holes(table, lengths, page, pages, seed):
    """Missing pages (-1, past the cache, the types' ends) in the rows: first, last, beside the borders of 128-key grains, some at random."""
    g, none = np.random.Generator(np.random.PCG64(seed)), [-1, pages, -2 ** 31, 2 ** 31 - 1]
    for b, n in enumerate(lengths):
        if n <= 0:
            continue
        last = (n - 1) // page
        at = {0, last} if b % 2 else set()
        at |= {int(x) for x in g.integers(0, last + 1, 4)} | {min(last, 128 * int(x) // page) for x in g.integers(1, max(2, n // 128), 3)}
        for i, p in enumerate(sorted(at)):
            table[b, p] = none[(i + b) % 4]


@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("dim,hk,page,order", [(64, 2, 16, "slots"), (64, 2, 24, "heads"), (128, 1, 48, "heads"), (128, 3, 7, "slots"),
                                               (256, 2, 16, "heads"), (224, 1, 30, "slots")])
@pytest.mark.parametrize("window,softcap,starts", [(0, 0.0, False), (700, 0.0, True), (1500, 20.0, False), (0, 5.0, True)])
def test_masks_holes_and_nan_in_cut_rows(kind, cache, dim, hk, page, order, window, softcap, starts):
    require_gpu()
    lengths = [2500, 1400, 0, 641, 3000, 130]
    first = [999, 0, 5, 641, 2990, -7] if starts else None
    say(f"attention {cache} {order} dim={dim} heads={hk} page={page} window={window} softcap={softcap} starts={starts}")
    pages = sum(-(-n // page) for n in lengths) + 3
    c = Cache(cache, order, pages, page, hk, dim, dim + page)
    table = tables(lengths, page, pages, 3)
    holes(table, lengths, page, pages, 5)
    hide(c, table, lengths, first, window)
    q = normal((len(lengths), 3 * hk, dim), kind, 5, 2.0)
    ws = workspace(c, len(lengths), 3 * hk, 3000, window)
    args = dict(starts=first, window=window, softcap=softcap)
    out, lse = attend(c, kind, q, table, lengths, 3000, ws, **args)
    check(c, kind, q, out, lse, table, lengths, **args)
    again = attend(c, kind, q, table, lengths, 3000, ws, **args)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse), "not deterministic"
    whole = attend(c, kind, q, table, lengths, 3000, **args)                     # no workspace: rows are not cut
    check(c, kind, q, *whole, table, lengths, **args)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim,page,hq,hk", [(200, 16, 12, 3), (248, 32, 2, 2), (256, 16, 40, 2), (256, 64, 16, 1), (136, 48, 5, 1)])
def test_large_heads_in_cut_rows(kind, dim, page, hq, hk):
    """16-bit heads above 128 elements in pages of whole half tiles, whose kernel keeps its queries in LDS."""
    require_gpu()
    lengths = [2049, 5000, 700]
    say(f"attention {kind} dim={dim} page={page} heads={hq}/{hk}")
    pages = sum(-(-n // page) for n in lengths)
    c = Cache(kind, "slots", pages, page, hk, dim, dim)
    table = tables(lengths, page, pages, 3)
    q = normal((3, hq, dim), kind, 5)
    out, lse = attend(c, kind, q, table, lengths, 5000, workspace(c, 3, hq, 5000))
    check(c, kind, q, out, lse, table, lengths)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_extreme_scores_in_cut_rows(kind):
    """Large scores of both signs, equal scores, and a cap far above the scores, over many shares."""
    require_gpu()
    say(f"attention {kind}: extreme scores, 1900 keys")
    c = Cache(kind, "heads", 120, 16, 2, 64, 4)
    table = tables([1900], 16, 120, 3)
    q = normal((1, 4, 64), kind, 5, sigma=100.0)
    ws = workspace(c, 1, 4, 1900)
    for scale, softcap in ((1.0, 0.0), (0.0, 0.0), (1.0, 50.0)):
        out, lse = attend(c, kind, q, table, [1900], 1900, ws, scale=scale, softcap=softcap)
        check(c, kind, q, out, lse, table, [1900], scale=scale, softcap=softcap)
    q = normal((1, 4, 64), kind, 5, sigma=3.0)
    for softcap in (1e6, 3e38):
        out, lse = attend(c, kind, q, table, [1900], 1900, ws, softcap=softcap)
        check(c, kind, q, out, lse, table, [1900])


def test_non_finite_values_in_cut_rows():
    """A NaN in an attended value spoils its element of its head, in whichever share; one in a key its head's rows."""
    require_gpu()
    say("attention: NaN in attended places of cut rows")
    c = Cache("f16", "heads", 120, 16, 2, 64, 4)
    table = tables([1900], 16, 120, 3)
    q, ws = normal((1, 4, 64), "f16", 5), workspace(c, 1, 4, 1900)
    clean = f64(attend(c, "f16", q, table, [1900], 1900, ws)[0])
    for j in (0, 127, 128, 1000, 1899):
        place = (int(table[0, j // 16]), 1, j % 16, 5)
        old = c.planes[1][place].clone()
        c.planes[1][place] = float("nan")
        out, lse = attend(c, "f16", q, table, [1900], 1900, ws)
        bad = np.isnan(f64(out))
        assert bad[0, 2:, 5].all() and bad.sum() == 2 and np.isfinite(f64(lse)).all(), j
        assert np.array_equal(f64(out)[~bad], clean[~bad])
        c.planes[1][place] = old
    c.planes[0][int(table[0, 60]), 0, 3, 3] = float("nan")
    out, lse = attend(c, "f16", q, table, [1900], 1900, ws)
    assert np.isnan(f64(out))[0, :2].all() and np.isnan(f64(lse))[0, :2].all() and np.isfinite(f64(lse))[0, 2:].all()


@pytest.mark.parametrize("kind,cache,dim,page", [("f16", "f16", 128, 16), ("bf16", "e4m3", 64, 24), ("bf16", "bf16", 96, 5), ("f16", "e4m3", 128, 32)])
@pytest.mark.parametrize("window,softcap,starts", [(0, 0.0, True), (64000, 10.0, False)])
def test_two_head_tiles_with_masks(kind, cache, dim, page, window, softcap, starts):
    """More than 16 query heads to a cache head and keys enough that two tiles of heads meet a key together (a workspace for 32
    heads a slot says so), with starts or a window and a cap, missing pages and NaN beside the attended keys. The rows share their pages."""
    require_gpu()
    n, hq = 66000, 20
    most = 256 if 2 * 128 * 2 * dim * (1 if cache == "e4m3" else 2) >= 131072 else 512      # workgroups with one tile of heads
    seqs = 5 if most == 256 else 10
    first = [(7 * i, 31, 400)[i % 3] for i in range(seqs)] if starts else None
    say(f"attention {cache}: {hq} heads of {dim}, {seqs} rows of {n}, window={window} softcap={softcap} starts={starts}")
    pages = -(-n // page) + 2
    c = Cache(cache, "heads", pages, page, 1, dim, 8)
    row = tables([n], page, pages, 3)
    holes(row, [n], page, pages, 6)
    lengths = [n, n - 129, n - 1000] + [n] * (seqs - 3)
    hide(c, np.repeat(row, seqs, 0), lengths, first, window)
    q = normal((seqs, hq, dim), kind, 5, 2.0)
    ws = workspace(c, seqs, hq, n, window)
    assert ws.numel() == COUNTERS + 2 * 512 * 32 * (dim + 2) * 4, "one tile of heads"
    args = dict(window=window, softcap=softcap)
    out, lse = attend(c, kind, q, np.repeat(row, seqs, 0), lengths, n, ws, starts=first, **args)
    for b in (0, 1, 2):
        check(c, kind, q[b:b + 1], out[b:b + 1], lse[b:b + 1], row, lengths[b:b + 1], starts=first and first[b:b + 1], **args)


@pytest.mark.parametrize("kind,cache,hq,hk,dim,page,lengths", [
    ("f16", "f16", 16, 4, 256, 64, [30] * 50), ("f16", "f16", 8, 8, 128, 64, [500] * 12), ("bf16", "e4m3", 4, 2, 64, 24, list(range(0, 300, 3))),
    ("f16", "f16", 4, 1, 128, 16, [1]), ("bf16", "bf16", 34, 1, 96, 16, [0, 0, 7, 0]), ("f16", "e4m3", 3, 3, 32, 5, [0])])
def test_bounds_far_above_the_lengths(kind, cache, hq, hk, dim, page, lengths):
    """max_len as the cache's capacity, as a captured step passes it, over short rows: the kernel of shares runs them."""
    require_gpu()
    say(f"attention {cache}: {len(lengths)} rows of up to {max(lengths)} keys of {hk} x {dim}, bound 32768")
    pages = sum(-(-n // page) for n in lengths) + 1
    c = Cache(cache, "slots", pages, page, hk, dim, 11)
    table = tables(lengths, page, pages, 3, cols=-(-32768 // page))
    q = normal((len(lengths), hq, dim), kind, 5)
    out, lse = attend(c, kind, q, table, lengths, 32768, workspace(c, len(lengths), hq, 32768))
    check(c, kind, q, out, lse, table, lengths)


@pytest.mark.parametrize("hk,lengths", [(1, [150000]), (1, [70000, 300, 60000]), (2, [40000, 90000]), (4, [3000] * 70)])
def test_counters_after_joins_of_every_depth(hk, lengths):
    """Joins in one step and in two, several a workgroup: attend() looks at all counters after each of three calls."""
    require_gpu()
    say(f"attention: joins of {hk} heads, rows of {lengths[:3]}")
    pages = sum(-(-n // 32) for n in lengths)
    c = Cache("f16", "heads", pages, 32, hk, 64, 8)
    table = tables(lengths, 32, pages, 3)
    q = normal((len(lengths), 2 * hk, 64), "f16", 5)
    ws = workspace(c, len(lengths), 2 * hk, max(lengths))
    got = [attend(c, "f16", q, table, lengths, max(lengths), ws) for _ in range(3)]
    check(c, "f16", q, *got[0], table, lengths)
    assert all(torch.equal(a, got[0][0]) and torch.equal(b, got[0][1]) for a, b in got[1:])
