"""A step's pages, tokens and slots on the device, against the same rules in plain Python."""
import numpy as np
import pytest
import torch

from gpu_common import dev, host, require_gpu, say

pytestmark = pytest.mark.gpu


def plan(page, cols, pages, max_tokens, table, lengths, wants, free, n_free, kept):
    """(table, lengths, stack, offsets, tokens, status) after the step; the stack as a list with its top at the end."""
    n = len(lengths)
    has = [min(max(x, 0), cols * page) for x in lengths]
    to = [h if w < 0 else w for h, w in zip(has, wants)]
    need = [(-(-h // page), -(-min(t, cols * page) // page)) for h, t in zip(has, to)]
    gives = [(b, c) for b in range(n) for c in range(need[b][1], need[b][0]) if c >= kept[b]]
    takes = [(b, c) for b in range(n) for c in range(need[b][0], need[b][1])]
    tokens = [(b, p) for b in range(n) for p in range(has[b], min(to[b], cols * page))]
    stack = list(free[:min(max(n_free, 0), pages)])
    status = (4 if any(t > cols * page for t in to) else 0) | (2 if len(tokens) > max_tokens else 0)
    status |= (1 if len(takes) > len(stack) + len(gives) else 0) | (8 if len(stack) + len(gives) > pages else 0)
    if status:
        return table, list(lengths), stack, [0] * (n + 1), [], status
    table = table.copy()
    stack += [table[b, c] for b, c in reversed(gives)]
    for b in range(n):
        table[b, need[b][1]:need[b][0]] = -1
    for b, c in takes:
        table[b, c] = stack.pop()
    offsets = np.concatenate([[0], np.cumsum([max(0, t - h) for h, t in zip(has, to)])]).tolist()
    return table, to, stack, offsets, tokens, 0


class Step:
    """The device's state and one call after another, each held against plan()."""

    def __init__(self, seqs, cols, page, pages, room, seed, slots=True):
        self.g = np.random.Generator(np.random.PCG64(seed))
        self.page, self.cols, self.pages, self.room = page, cols, pages, room
        self.table, self.lengths = np.full((seqs, cols), -1, np.int32), [0] * seqs
        self.stack = self.g.permutation(pages).astype(np.int32).tolist()
        self.d_table, self.d_lengths = dev(self.table), dev(np.zeros(seqs, np.int32))
        self.d_free, self.d_n = dev(np.array(self.stack, np.int32)), dev(np.array([pages], np.int32))
        self.d_offsets, self.d_status = (torch.full((k,), 77, dtype=torch.int32, device="cuda") for k in (seqs + 1, 1))
        self.maps = [torch.full((room,), 77, dtype=torch.int32, device="cuda") for _ in range(3)]
        if not slots:
            self.maps[2] = None

    def call(self, wants, kept=None, in_place=True):
        api = require_gpu()
        n = len(self.lengths)
        want = plan(self.page, self.cols, self.pages, self.room, self.table, self.lengths, wants, np.array(self.stack, np.int32), len(self.stack), kept or [0] * n)
        d_kept = None if kept is None else dev(np.array(kept, np.int32))
        new = (None, None) if in_place else (torch.full_like(self.d_lengths, 77), torch.full_like(self.d_n, 77))
        api.mxkv_step_run(self.page, self.d_table, self.d_lengths, dev(np.array(wants, np.int32)), self.d_free, self.d_n, self.d_offsets, *self.maps,
                          self.d_status, kept=d_kept, lengths_out=new[0], n_free_out=new[1])
        if not in_place:
            torch.cuda.synchronize()
            assert host(self.d_lengths).tolist() == self.lengths and host(self.d_n).tolist() == [len(self.stack)]
            self.d_lengths, self.d_n = new
        self.table, self.lengths, self.stack, offsets, tokens, status = want
        assert host(self.d_status).tolist() == [status]
        assert np.array_equal(host(self.d_table), self.table)
        assert host(self.d_lengths).tolist() == list(self.lengths)
        assert host(self.d_n).tolist() == [len(self.stack)]
        assert host(self.d_free)[:len(self.stack)].tolist() == [int(p) for p in self.stack]
        assert host(self.d_offsets).tolist() == offsets
        more = self.room - len(tokens)
        assert host(self.maps[0]).tolist() == [b for b, _ in tokens] + [-1] * more
        assert host(self.maps[1]).tolist() == [p for _, p in tokens] + [-1] * more
        if self.maps[2] is not None:
            assert host(self.maps[2]).tolist() == [int(self.table[b, p // self.page]) * self.page + p % self.page for b, p in tokens] + [-1] * more
        return status


@pytest.mark.parametrize("seqs,cols,page,pages,room", [(1, 1, 1, 1, 4), (3, 5, 4, 20, 64), (64, 40, 16, 1500, 3000), (7, 30, 37, 100, 8192), (1024, 6, 16, 5000, 8192),
                                                       (1025, 9, 8, 6000, 20000), (2500, 4, 7, 6000, 9000), (5, 900, 16, 3000, 60000)])
def test_random_steps(seqs, cols, page, pages, room):
    """Rows grow, shrink, end, stay; some steps are refused and change nothing."""
    s = Step(seqs, cols, page, pages, room, seqs + room)
    seen = set()
    for i in range(10):
        most = cols * page
        grow = s.g.integers(0, max(2, min(most, 2 * room // seqs + 2)), seqs)
        wants = [int(min(most, max(0, n + (x if a < 0.6 else 0 if a < 0.75 else -x)))) for n, x, a in zip(s.lengths, grow, s.g.random(seqs))]
        wants = [w if a < 0.9 else -1 if a < 0.95 else 0 for w, a in zip(wants, s.g.random(seqs))]
        seen.add(s.call(wants, in_place=i % 2 == 0))
    say(f"{seqs} rows of {cols} x {page}: statuses {sorted(seen)}")


@pytest.mark.parametrize("seqs", [4, 1500])
def test_refusals_on_the_device(seqs):
    """Each reason alone and together, with the state as it was."""
    s = Step(seqs, 8, 4, 3 * seqs, 2 * seqs, 1)
    assert s.call([1] * seqs) == 0
    assert s.call([3] * seqs) == 0
    assert s.call([32] + [4] * (seqs - 1)) == 0 if seqs > 50 else True
    assert s.call([33] + [-1] * (seqs - 1)) & 4
    assert s.call([32] * seqs) & 3 == 3
    s.room_before = s.room
    assert s.call([s.lengths[0]] + [-1] * (seqs - 1)) == 0


@pytest.mark.parametrize("seqs", [1024, 1025, 2100, 3000])
def test_sums_past_32_bits(seqs):
    """Rows that together want more tokens and pages than 32 bits count: refused, and nothing changes."""
    api = require_gpu()
    page, cols, pages = 2, 540000, 7
    full = lambda n, v: torch.full((n,), v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((seqs, cols), -1, dtype=torch.int32, device="cuda")
    lengths, free, n_free, status, offsets = full(seqs, 0), torch.arange(pages, dtype=torch.int32, device="cuda"), full(1, pages), full(1, 77), full(seqs + 1, 77)
    maps = [full(16, 77) for _ in range(3)]
    say(f"{seqs} rows that want all of {cols} pages")
    api.mxkv_step_run(page, table, lengths, full(seqs, page * cols), free, n_free, offsets, *maps, status)
    torch.cuda.synchronize()
    assert status.item() == api.MXKV_STEP_PAGES | api.MXKV_STEP_TOKENS
    assert not lengths.any() and n_free.item() == pages and not offsets.any() and bool((table == -1).all()) and all(bool((m == -1).all()) for m in maps)


def test_stack_that_is_not_free():
    """A stack that says it is full while rows hold pages is not written past its end."""
    s = Step(2, 4, 2, 8, 16, 1)
    s.call([8, 8])
    s.d_n.fill_(8)
    s.stack = host(s.d_free).tolist()
    assert s.call([0, 0]) == 8


def test_given_back_is_restored():
    s = Step(50, 30, 16, 1200, 9000, 3)
    s.call(s.g.integers(0, 100, 50).tolist())
    before = (s.table.copy(), list(s.lengths), list(s.stack))
    s.call([n + int(x) for n, x in zip(s.lengths, s.g.integers(0, 200, 50))])
    s.call(before[1])
    assert np.array_equal(s.table, before[0]) and s.lengths == before[1] and s.stack == before[2]


def test_kept_pages():
    """Columns that a row shares leave its table when it ends, and do not come to the stack."""
    s = Step(6, 10, 4, 60, 400, 4)
    s.call([8, 8, 8, 8, 0, 0])
    kept = [0, 1, 2, 5, 0, 3]
    s.call([0, 0, 0, 0, 9, 3], kept=kept)
    s.call([5, 1, 0, 2, 1, 0], kept=kept)
    s.call([0] * 6, kept=[1, 0, 0, 1, 0, 1])


def test_without_slots_and_tokens():
    s = Step(9, 5, 16, 40, 30, 5, slots=False)
    s.call([3] * 9)
    s.call([5, 0] + [-1] * 7)
    z = Step(4, 5, 16, 40, 0, 6)
    z.call([0, -1, 0, 0])
    assert z.call([1, 0, 0, 0]) == 2


def test_missing_pages_have_no_slots():
    """Entries of the stack that are no pages go into the table, and their tokens get no slot."""
    api = require_gpu()
    s = Step(1, 3, 4, 4, 12, 1)
    s.d_free.copy_(dev(np.array([2, 9, -5, 1], np.int32)))
    api.mxkv_step_run(4, s.d_table, s.d_lengths, dev(np.array([12], np.int32)), s.d_free, s.d_n, s.d_offsets, *s.maps, s.d_status)
    assert host(s.d_table).tolist() == [[1, -5, 9]]
    assert host(s.maps[2]).tolist() == [4, 5, 6, 7] + [-1] * 8


def test_graph_of_decode_steps():
    """A captured step of one token per row, replayed: the lengths go on by themselves."""
    api = require_gpu()
    s = Step(5, 8, 2, 40, 8, 7)
    s.call([3, 0, 1, 4, 2][:5])
    wants = torch.zeros(5, dtype=torch.int32, device="cuda")
    table, stack, lengths = s.table.copy(), list(s.stack), list(s.lengths)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        torch.add(s.d_lengths, 1, out=wants)
        api.mxkv_step_run(2, s.d_table, s.d_lengths, wants, s.d_free, s.d_n, s.d_offsets, *s.maps, s.d_status)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        table, lengths, stack, _, tokens, status = plan(2, 8, 40, 8, table, lengths, [n + 1 for n in lengths], np.array(stack, np.int32), len(stack), [0] * 5)
        assert status == 0 and host(s.d_lengths).tolist() == lengths and np.array_equal(host(s.d_table), table)
        assert host(s.maps[0]).tolist() == [0, 1, 2, 3, 4, -1, -1, -1]


def test_rows_of_a_step_are_appended():
    """The maps drive mxkv_append_run: every token lands in its slot, and the places behind the last one write nothing."""
    api = require_gpu()
    s = Step(3, 4, 4, 12, 16, 8)
    s.call([5, 0, 2])
    s.call([9, 1, 5])
    k, v = (torch.randn(16, 2, 32, generator=torch.Generator().manual_seed(i)).half().cuda() for i in (1, 2))
    planes = [torch.zeros(12, 4, 2, 32, dtype=torch.float16, device="cuda") for _ in range(2)]
    cache = api.KVCache(api.MX_F16, *planes, order=api.MXKV_SLOTS_FIRST)
    api.mxkv_append_run(cache, api.MX_F16, k, v, s.maps[1], s.d_table, seq=s.maps[0])
    slots = host(s.maps[2])
    for plane, x in zip(planes, (k, v)):
        want = torch.zeros(48, 2, 32, dtype=torch.float16, device="cuda")
        for t, slot in enumerate(slots):
            if slot >= 0:
                want[int(slot)] = x[t]
        assert torch.equal(plane.view(48, 2, 32), want)
