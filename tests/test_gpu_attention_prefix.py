"""Attention of a batch whose rows share beginnings, every row against the formula over its whole length."""
import numpy as np
import pytest
import torch

from attention_common import check, hide
from cache_common import Cache, fmt_of, normal
from gpu_common import dev, require_gpu, say

pytestmark = pytest.mark.gpu
COUNTERS = 3 * 512 * 4
FAR = 1 << 22   # bounds that are far above the lengths, for which the call shares whatever little there is


class Batch:
    """Groups of rows: their tables begin with the pages of shared[g] positions, and go on with pages of their own."""

    def __init__(self, kind, cache, order, dim, page, heads, share, members, shared, own, seed=0, outside=(0, 0), extra=3):
        g = np.random.Generator(np.random.PCG64(seed))
        self.kind, self.share = kind, share
        n = sum(members) + sum(outside)
        self.first = np.concatenate([[0], np.cumsum(members)]).astype(np.int32) + outside[0]
        self.shared = np.array(shared, np.int32)
        own = list(own) if hasattr(own, "__len__") else g.integers(0, own + 1, n).tolist()
        group = np.searchsorted(self.first, np.arange(n), side="right") - 1
        whole = [s // page if 0 <= i < len(shared) and self.first[i] <= b < self.first[i + 1] else 0
                 for b, i in enumerate(group) for s in [shared[i] if 0 <= i < len(shared) else 0]]
        self.lengths = np.array([w * page + o for w, o in zip(whole, own)], np.int32)
        need = [-(-o // page) for o in own]
        pages = sum(s // page for s in shared) + sum(need) + extra
        order_of = g.permutation(pages).astype(np.int32)
        self.table = np.full((n, max(1, max(w + x for w, x in zip(whole, need)))), -1, np.int32)
        at = 0
        for i, s in enumerate(shared):
            common = order_of[at:at + s // page]
            at += len(common)
            for b in range(self.first[i], self.first[i + 1]):
                self.table[b, :len(common)] = common
        for b in range(n):
            self.table[b, whole[b]:whole[b] + need[b]] = order_of[at:at + need[b]]
            at += need[b]
        self.c = Cache(cache, order, pages, page, heads, dim, seed + 1)
        self.q = normal((n, heads * share, dim), kind, seed + 2)

    def run(self, softcap=0.0, max_len=None, max_shared=None, sharing=True, ws=None, shared=None):
        api = require_gpu()
        n, hq, dim = self.q.shape
        max_len = max_len or FAR
        shared = self.shared if shared is None else np.array(shared, np.int32)
        most = FAR if max_shared is None else max_shared
        need = api.mxattn_prefix_workspace_size(self.c.c, n, hq, len(shared), max_len, most)
        if ws is None:
            ws = torch.full((max(16, need),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever nothing is written
            ws[:COUNTERS] = 0
        out, lse = torch.full(self.q.shape, float("nan"), dtype=self.q.dtype, device="cuda"), torch.full((n, hq), 99.0, device="cuda")
        say(f"{n} rows of {hq} heads, groups {len(shared)}, dim {dim}, workspace {need}")
        api.mxattn_prefix_run(self.c.c, fmt_of(api, self.kind), self.q, out, dev(self.table), dev(self.lengths), max_len, dev(self.first), dev(shared), most,
                              dim ** -0.5, lse=lse, softcap=softcap, workspace=ws if sharing else None)
        torch.cuda.synchronize()
        assert not bool(ws[:COUNTERS].any()), "counters not back at zero"
        return out, lse

    def check(self, out, lse, softcap=0.0):
        check(self.c, self.kind, self.q, out, lse, self.table, self.lengths, softcap=softcap)


@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("order", ["heads", "slots"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 16), (96, 24), (32, 7), (160, 33)])
def test_types(kind, cache, order, dim, page):
    b = Batch(kind, cache, order, dim, page, 2, 3, [3, 5], [300, 200], 50)
    hide(b.c, b.table, b.lengths)
    b.check(*b.run())


@pytest.mark.parametrize("dim", [8, 40, 72, 120, 136, 248])
def test_odd_head_sizes(dim):
    b = Batch("f16", "f16", "slots", dim, 16, 3, 5, [4], [400], 30)
    hide(b.c, b.table, b.lengths)
    b.check(*b.run())


@pytest.mark.parametrize("share,members", [(1, [2]), (1, [70]), (7, [40]), (16, [9]), (20, [13]), (8, [64, 2, 33])])
def test_rows_of_tiles(share, members):
    """Groups of fewer rows than a wave has, of several tiles, of heads that two tiles of the second launch take."""
    b = Batch("bf16", "bf16", "heads", 64, 16, 2, share, members, [200] * len(members), 40)
    b.check(*b.run())


@pytest.mark.parametrize("members,shared,own,outside", [
    ([4], [63], 40, (0, 0)),                             # less than a tile
    ([4], [64], 40, (0, 0)),
    ([1, 1, 3], [500, 300, 400], 40, (0, 0)),            # single rows
    ([2, 3], [128, 256], 40, (2, 3)),                    # rows in no group
    ([2, 0, 3], [128, 0, 192], 40, (0, 0)),              # an empty group
    ([5], [0], 90, (0, 0)),
    ([3], [640], [0, 0, 0], (0, 0)),                     # rows that share all they have
])
def test_groups(members, shared, own, outside):
    b = Batch("f16", "f16", "heads", 128, 16, 2, 4, members, shared, own, outside=outside)
    hide(b.c, b.table, b.lengths)
    b.check(*b.run())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_short_and_empty_rows(cache):
    """Rows that end before their group's beginning does, and rows without positions, wherever they are in the group."""
    b = Batch("bf16", cache, "slots", 128, 16, 2, 4, [4, 3, 2], [512, 320, 200], 30)
    b.lengths[[0, 5, 7, 8]] = [0, 100, 0, 0]
    b.check(*b.run())
    b.lengths[:] = 0
    out, lse = b.run(max_len=600)
    assert not out.any() and bool((lse == -float("inf")).all())


def test_shared_through_the_first_row():
    """What a group shares is what its first sequence's row names."""
    b = Batch("f16", "f16", "heads", 64, 16, 2, 2, [3], [320], 40)
    want = b.table.copy()
    b.table[1:, :20] = -1
    out, lse = b.run()
    b.table = want
    b.check(out, lse)


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_rows_that_have_ended(cache):
    """A group goes on when its first rows end: rows without positions, whose tables name no pages, do not count."""
    b = Batch("f16", cache, "heads", 128, 16, 2, 4, [4, 3, 2], [512, 320, 256], 40, outside=(1, 1))
    for row in (1, 2, 5, 8):
        b.lengths[row], b.table[row] = 0, -1
    b.check(*b.run())


def test_missing_pages():
    """Positions whose page is missing are left out, in what is shared too; a whole group may have none."""
    b = Batch("f16", "f16", "heads", 128, 16, 2, 4, [3, 2], [512, 256], 40)
    b.table[:3, [0, 3, 4, 5, 6, 7, 31]] = [-1, 99999, -1, -1, -1, -1, -5]
    b.table[3:] = -1
    b.check(*b.run())


@pytest.mark.parametrize("softcap", [2.0, 30.0, 1e30])
@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_softcap(softcap, cache):
    b = Batch("f16", cache, "heads", 128, 32, 2, 6, [5], [300], 50)
    b.check(*b.run(softcap=softcap), softcap=softcap)


@pytest.mark.parametrize("kind,cache,dim", [("f16", "f16", 128), ("bf16", "bf16", 128), ("f16", "e4m3", 128), ("bf16", "bf16", 256), ("f16", "f16", 64)])
def test_long(kind, cache, dim):
    """Long beginnings, split among workgroups, and rows of their own that are cut as well."""
    b = Batch(kind, cache, "heads", dim, 64, 1, 8, [6, 3], [20000, 9000], 3000)
    b.check(*b.run())


def test_many_groups():
    """More groups than threads, of two rows each; more work items than workgroups."""
    b = Batch("f16", "f16", "slots", 64, 16, 4, 1, [2] * 300, [64 + 16 * (i % 20) for i in range(300)], 20)
    b.check(*b.run())


@pytest.mark.parametrize("cache,dim", [("e4m3", 128), ("f16", 256)])
def test_most_groups(cache, dim):
    """As many groups as there may be, whose lists need the most LDS; some have one row, or none."""
    b = Batch("f16", cache, "heads", dim, 16, 1, 1, [i % 4 for i in range(1024)], [64 + 64 * (i % 2) for i in range(1024)], 9)
    b.check(*b.run())


def test_bounds():
    """shared above max_shared is taken as it, lengths above max_len too; bounds far above both change nothing."""
    b = Batch("f16", "f16", "heads", 128, 16, 2, 4, [4], [600], 40)
    for most in (1, 64, 100, 1 << 20):
        b.check(*b.run(max_shared=most))
    b.check(*b.run(max_len=int(b.lengths.max()), max_shared=600))
    b.check(*b.run(shared=[1 << 30]))
    b.check(*b.run(shared=[-7]))
    full = b.lengths.copy()
    out, lse = b.run(max_len=500)
    b.lengths = np.minimum(full, 500)
    b.check(out, lse)


def test_falling_firsts_share_nothing():
    b = Batch("f16", "f16", "heads", 64, 16, 2, 2, [3, 2], [320, 320], 40)
    for first in ([0, 5, 2], [4, 0, 5], [-9, 99, 3]):
        b.first = np.array(first, np.int32)
        b.check(*b.run())


def test_little_to_share():
    """Where the bounds leave less to share than a pass of its own costs, every row is read by itself."""
    b = Batch("f16", "f16", "heads", 128, 16, 2, 4, [4, 3], [600, 300], 40)
    api, n, hq = require_gpu(), *b.q.shape[:2]
    assert api.mxattn_prefix_workspace_size(b.c.c, n, hq, 2, 700, 600) == api.mxattn_decode_workspace_size(b.c.c, n, hq, 700)
    b.check(*b.run(max_len=700, max_shared=600))


def test_without_workspace():
    b = Batch("f16", "f16", "heads", 128, 16, 2, 4, [4, 3], [600, 300], 40)
    b.check(*b.run(sharing=False))
    b.check(*b.run(ws=torch.zeros(COUNTERS + 16, dtype=torch.uint8, device="cuda")))


def test_one_workspace_for_all():
    """Batches of several shapes and the decode call use one buffer in turn."""
    api = require_gpu()
    ws = torch.zeros(256 << 20, dtype=torch.uint8, device="cuda")
    batches = [Batch("f16", "f16", "heads", 128, 16, 2, 4, [4, 3], [6000, 300], 400), Batch("bf16", "e4m3", "slots", 64, 32, 3, 2, [9], [1000], 900),
               Batch("f16", "f16", "heads", 256, 16, 1, 9, [20], [500], 4000)]
    for _ in range(2):
        for b in batches:
            b.check(*b.run(ws=ws))
            out, lse = torch.empty_like(b.q), torch.empty(b.q.shape[:2], device="cuda")
            api.mxattn_decode_run(b.c.c, fmt_of(api, b.kind), b.q, out, dev(b.table), dev(b.lengths), int(b.lengths.max()), b.q.shape[2] ** -0.5, lse=lse, workspace=ws)
            b.check(out, lse)


def test_infinite_scores_and_nan_queries():
    """NaN where the rows by themselves give it: queries with NaN, of rows that share all they have too, and scores that are infinite, which softmax
    makes NaN (a score of -infinity counts nothing)."""
    b = Batch("f16", "f16", "heads", 128, 16, 2, 4, [3, 2], [320, 256], [0, 30, 0, 20, 0])
    b.q[0, 3, 7] = b.q[1, 5, 0] = float("nan")
    b.c.planes[0][int(b.table[3, 2]), 1, 3, 9] = float("inf")
    b.q[3, 4, 9], b.q[3, 5, 9], b.q[4, 4, 9], b.q[4, 5, 9] = 1.0, -1.0, -1.0, 1.0
    (out, lse), (want, want_lse) = b.run(), b.run(sharing=False)
    for row, head, bad in ((0, 3, True), (1, 5, True), (2, 5, False), (3, 4, True), (3, 5, False), (4, 4, False), (4, 5, True)):
        assert bool(want[row, head].isnan().all()) == bool(want[row, head].isnan().any()) == bad
    assert torch.equal(out.isnan(), want.isnan()) and torch.equal(lse.isnan(), want_lse.isnan())
    # two results off by half a step of binary16, and by what the sums lose, each
    assert ((out - want).abs().nan_to_num() <= 4 * 2.0 ** -11 * want.abs().nan_to_num().max()).all()


def test_infinite_values_and_nan():
    """A shared value that is infinite or NaN reaches every row of the group and no other row."""
    for bad in (float("inf"), float("nan")):
        b = Batch("f16", "f16", "slots", 64, 16, 1, 2, [3, 2], [320, 128], 40)
        page = int(b.table[0, 2])
        b.c.planes[1][page, 3, 0, 5] = bad
        out, _ = b.run()
        bad_at = ~torch.isfinite(out)
        assert bool(bad_at[:3, :, 5].all()) and int(bad_at.sum()) == 6
        assert bool((out[:3, :, 5] == bad).all()) if bad == float("inf") else bool(out[:3, :, 5].isnan().all())


def test_strides_and_streams():
    """Queries and outputs as slices of wider tensors, on another stream."""
    api = require_gpu()
    b = Batch("f16", "f16", "heads", 64, 16, 2, 3, [4], [300], 40)
    wide = torch.randn(4, 10, 64, generator=torch.Generator().manual_seed(5)).half().cuda()
    b.q = wide[:, 2:8]
    n, hq, dim = b.q.shape
    out_wide = torch.full((4, 9, 72), float("nan"), dtype=torch.float16, device="cuda")
    out, lse = out_wide[:, 1:7, :64], torch.zeros(n, hq, device="cuda")
    need = api.mxattn_prefix_workspace_size(b.c.c, n, hq, 1, FAR, FAR)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    args = [dev(t) for t in (b.table, b.lengths, b.first, b.shared)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    api.mxattn_prefix_run(b.c.c, api.MX_F16, b.q, out, args[0], args[1], FAR, args[2], args[3], FAR, dim ** -0.5, lse=lse, workspace=ws, stream=stream)
    stream.synchronize()
    b.check(out, lse)
    assert int(out_wide.isnan().sum()) == out_wide.numel() - out.numel()


def test_graph():
    """Captured, and replayed with other lengths, groups and queries."""
    api = require_gpu()
    b = Batch("f16", "f16", "heads", 128, 16, 2, 4, [4, 3], [600, 300], 200)
    n, hq, dim = b.q.shape
    out, lse = torch.zeros_like(b.q), torch.zeros(n, hq, device="cuda")
    ws = torch.zeros(api.mxattn_prefix_workspace_size(b.c.c, n, hq, 2, FAR, FAR), dtype=torch.uint8, device="cuda")
    table, lengths, first, shared = (dev(t) for t in (b.table, b.lengths, b.first, b.shared))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.mxattn_prefix_run(b.c.c, api.MX_F16, b.q, out, table, lengths, FAR, first, shared, FAR, dim ** -0.5, lse=lse, workspace=ws)
    full = b.lengths.copy()
    for i, (new_shared, cut) in enumerate((([600, 300], 0), ([0, 128], 3), ([592, 64], 50), ([600, 300], 0))):
        b.lengths = np.maximum(full - cut, 0).astype(np.int32)
        lengths.copy_(dev(b.lengths))
        shared.copy_(dev(np.array(new_shared, np.int32)))
        b.q.copy_(normal(tuple(b.q.shape), "f16", 50 + i))
        graph.replay()
        torch.cuda.synchronize()
        b.check(out, lse)
        assert not bool(ws[:COUNTERS].any())


def test_deterministic():
    b = Batch("bf16", "bf16", "slots", 128, 16, 4, 8, [20, 30], [3000, 2000], 300)
    first = b.run()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, b.run()))


@pytest.mark.parametrize("kind,cache,dim,heads", [("f16", "f16", 40, 12), ("bf16", "e4m3", 64, 12), ("bf16", "bf16", 72, 12), ("f16", "e4m3", 96, 12), ("f16", "f16", 136, 6),
                                                  ("bf16", "e4m3", 160, 6)])
def test_many_tiles(kind, cache, dim, heads):
    """Workgroups with more tiles than they look up the pages of at a time, which end one unit and begin another."""
    b = Batch(kind, cache, "heads", dim, 16, heads, 1, [2], [20000], 20)
    b.check(*b.run())
