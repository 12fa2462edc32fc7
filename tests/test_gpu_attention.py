"""Attention of one new token over a paged cache against the formula in 64 bits."""
import numpy as np
import pytest
import torch

import cache_reference as ref
from cache_common import TORCH, Cache, f64, fmt_of, normal, tables
from gpu_common import dev, host, require_gpu, say

pytestmark = pytest.mark.gpu


def run(api, c, kind, q, table, lengths, max_len, split=True, starts=None, window=0, softcap=0.0, scale=None, out=None, ws=None):
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full(q.shape[:2], 99.0, device="cuda")
    if split and ws is None:
        need = api.mxattn_decode_workspace_size(c.c, q.shape[0], q.shape[1], max_len, window)
        ws = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")
    api.mxattn_decode_run(c.c, fmt_of(api, kind), q, out, dev(table), dev(np.asarray(lengths, np.int32)), max_len,
                          q.shape[2] ** -0.5 if scale is None else scale, lse=lse,
                          starts=None if starts is None else dev(np.asarray(starts, np.int32)), window=window, softcap=softcap,
                          workspace=ws if split else None)
    if split and ws is not None and ws.numel() > 16:
        torch.cuda.synchronize()
        counters = 4 * q.shape[0] * c.heads * -(-(q.shape[1] // c.heads) // 16)
        assert not bool(ws[:counters].any()), "counters not back at zero"
    return out, lse


def check(c, kind, q, out, lse, table, lengths, starts=None, window=0, softcap=0.0, scale=None):
    q64, o64, l64 = f64(q), f64(out), f64(lse)
    n, hq, dim = q64.shape
    share = hq // c.heads
    scale = float(np.float32(dim ** -0.5 if scale is None else scale))
    worst = [0.0, 0.0]
    for b in range(n):
        hi = max(0, min(lengths[b], table.shape[1] * c.page))
        lo = max(0, starts[b]) if starts is not None else 0
        lo = max(lo, hi - window) if window else lo
        k, ok = ref.gather(c.k, table[b], hi, c.page, c.order)
        v, _ = ref.gather(c.v, table[b], hi, c.page, c.order)
        ok &= np.arange(hi) >= lo
        for h in range(c.heads):
            at = slice(h * share, (h + 1) * share)
            want, wl, eo, el, spread = ref.attention(q64[b, at], k[h][ok], v[h][ok], scale, softcap)
            # the probabilities' rounding, the result's, and what 16 bits cannot hold
            bound = eo + ref.HALF_STEP[kind] * (spread + np.abs(want)) * (1 + 2.0 ** -6) + ref.TINY[kind]
            empty = not ok.any()
            if empty:
                assert not o64[b, at].any() and np.all(l64[b, at] == -np.inf), (b, h)
                continue
            err = np.abs(o64[b, at] - want) / bound
            worst = [max(worst[0], err.max()), max(worst[1], (np.abs(l64[b, at] - wl) / el).max())]
            assert np.all(np.isfinite(o64[b, at])), (b, h)
    say(f"worst error / bound: out {worst[0]:.3f}, lse {worst[1]:.3f}")
    assert worst[0] <= 1.0 and worst[1] <= 1.0, worst


SHAPES = [  # q heads, heads, dim, page, lengths
    (1, 1, 8, 1, [1]), (4, 1, 32, 16, [0, 1, 2]), (12, 4, 64, 5, [31, 32, 33, 64]), (32, 8, 128, 16, [500, 17, 0, 128, 129]),
    (20, 1, 96, 24, [257, 1000]), (64, 4, 128, 64, [700, 64]), (6, 6, 256, 32, [300, 5]), (3, 3, 160, 7, [95, 96, 97]), (40, 2, 224, 100, [1500]),
    (2, 2, 64, 256, [5000, 3])]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("order", ["heads", "slots"])
@pytest.mark.parametrize("hq,hk,dim,page,lengths", SHAPES)
def test_attention(kind, quant, order, hq, hk, dim, page, lengths):
    api = require_gpu()
    if quant and dim % 32:
        dim = 32
    say(f"attention {kind} quant={quant} {order} heads={hq}/{hk} dim={dim} page={page} lengths={lengths}")
    pages = sum(-(-n // page) for n in lengths) + 2
    c = Cache("e4m3" if quant else kind, order, pages, page, hk, dim, hq + dim)
    table = tables(lengths, page, pages, 3)
    q = normal((len(lengths), hq + 2, dim), kind, 5)[:, 1:hq + 1]
    room = torch.full((len(lengths), hq, dim + 8), 5.0, dtype=q.dtype, device="cuda")
    for split in (True, False):
        out, lse = run(api, c, kind, q, table, lengths, max(1, max(lengths)), split=split, out=room[..., :dim])
        check(c, kind, q, out, lse, table, lengths)
        assert bool((room[..., dim:] == 5.0).all())
    again, lse2 = run(api, c, kind, q, table, lengths, max(1, max(lengths)), split=False)
    assert torch.equal(again, out) and torch.equal(lse2, lse), "not deterministic"


@pytest.mark.parametrize("dim", [72, 80, 112, 200, 248])
def test_attention_odd_head_sizes(dim):
    api = require_gpu()
    say(f"attention dim={dim}")
    c = Cache("f16", "heads", 30, 16, 2, dim, dim, paired=True)
    table = tables([300, 37], 16, 30, 3)
    q = normal((2, 6, dim), "f16", 5)
    out, lse = run(api, c, "f16", q, table, [300, 37], 300)
    check(c, "f16", q, out, lse, table, [300, 37])


@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("window,softcap,starts", [(1, 0.0, None), (33, 0.0, None), (1000, 5.0, None), (0, 30.0, [0, 100, 699, 700, 9999]),
                                                   (64, 0.0, [650, -3, 0, 31, 32]), (0, 0.0, [33, 64, 1, 260, 500])])
def test_attention_masks(kind, cache, window, softcap, starts):
    api = require_gpu()
    say(f"attention {cache} window={window} softcap={softcap} starts={starts}")
    lengths = [700, 700, 700, 700, 513]
    c = Cache(cache, "slots", 5 * 44, 16, 2, 64, 9)
    table = tables(lengths, 16, 220, 3)
    q = normal((5, 8, 64), kind, 5, sigma=3.0)
    for split in (True, False):
        out, lse = run(api, c, kind, q, table, lengths, 700, split=split, starts=starts, window=window, softcap=softcap)
        check(c, kind, q, out, lse, table, lengths, starts, window, softcap)


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_attention_ignores_what_is_masked(cache):
    """NaN in every slot that is not attended, and page numbers outside the cache: positions behind them are
    left out, as the 64-bit form leaves them out."""
    api = require_gpu()
    say(f"attention {cache}: NaN in masked places, bad pages")
    lengths, starts, page = [300, 45, 64, 90], [17, 0, 64, 0], 16
    c = Cache(cache, "heads", 60, page, 3, 96, 4)
    table = tables(lengths, page, 40, 3, cols=20)
    table[0, 3], table[0, 10], table[3, 0] = 60, -7, 2 ** 31 - 1
    table[3, 5] = -2 ** 31
    seen = np.zeros((60, page), bool)
    for b, n in enumerate(lengths):
        j = np.arange(starts[b], n)
        p = table[b][j // page]
        ok = (p >= 0) & (p < 60)
        seen[p[ok], j[ok] % page] = True
    hide = torch.from_numpy(~seen).cuda()
    for t, s in zip(c.planes, c.scales):
        if cache == "e4m3":
            t.swapaxes(1, 2)[hide] = 0x7F
            s.swapaxes(1, 2)[hide] = 0xFF
        else:
            t.swapaxes(1, 2)[hide] = float("nan")
    q = normal((4, 6, 96), "f16", 5)
    for split in (True, False):
        out, lse = run(api, c, "f16", q, table, lengths, 300, split=split, starts=starts)
        check(c, "f16", q, out, lse, table, lengths, starts)


def test_attention_lengths_out_of_range():
    """Lengths above max_len or the table's width are cut to it, negative ones are empty."""
    api = require_gpu()
    c = Cache("f16", "heads", 20, 16, 1, 64, 4)
    table = tables([160, 160], 16, 20, 3)
    q = normal((2, 2, 64), "f16", 5)
    say("attention: lengths out of range")
    out, lse = run(api, c, "f16", q, table, [2 ** 31 - 1, -5], 150)
    check(c, "f16", q, out, lse, table, [150, 0])
    out, lse = run(api, c, "f16", q, table, [2 ** 31 - 1, 161], 5000)
    check(c, "f16", q, out, lse, table, [160, 160])


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_attention_decodes_every_code_and_scale(kind):
    """One position: out is that position's value. Every E4M3 code at every scale code, where f holds the
    product without rounding; NaN codes and scales give NaN."""
    api = require_gpu()
    say(f"attention {kind}: every code and scale")
    seqs, heads, dim = 256, 8, 32                                     # sequence s: scale code s, head h: codes 32 h ..
    codes = np.broadcast_to(np.arange(256, dtype=np.uint8).reshape(1, heads, 1, dim), (seqs, heads, 1, dim)).copy()
    scales = np.broadcast_to(np.arange(256, dtype=np.uint8).reshape(seqs, 1, 1, 1), (seqs, heads, 1, 1)).copy()
    key = np.zeros_like(codes), np.full_like(scales, 127)
    c = api.KVCache(api.MX_E4M3, dev(key[0]), dev(codes), dev(key[1]), dev(scales))
    q = normal((seqs, heads, dim), kind, 1)
    out = torch.empty_like(q)
    api.mxattn_decode_run(c, fmt_of(api, kind), q, out, dev(np.arange(seqs, dtype=np.int32).reshape(-1, 1)),
                          dev(np.ones(seqs, np.int32)), 1, 1.0)
    want = np.zeros((seqs * heads, dim), np.float32)
    api.mx_unpack_host(api.MX_E4M3, codes, scales, seqs * heads, dim, want)
    want = want.reshape(seqs, heads, dim).astype(np.float64)
    got = f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    size = np.abs(np.nan_to_num(want))
    lo, hi = (2.0 ** -14, 65504.0) if kind == "f16" else (2.0 ** -100, 2.0 ** 100)  # 2^15 is held beside the value
    fits = (size >= lo) & (size <= hi) & ~np.isnan(want) | (want == 0)
    assert fits.sum() > 5000 and np.array_equal(got[fits], want[fits])


def test_attention_scores_use_every_key_element():
    """One-hot queries: the scores are single key elements, each of its own value, so a wrong order of the
    head's elements or of the keys shows at once."""
    api = require_gpu()
    say("attention: one-hot queries")
    for dim, cache in ((64, "f16"), (128, "f16"), (256, "f16"), (128, "e4m3"), (256, "e4m3"), (64, "e4m3")):
        c = Cache(cache, "heads", 4, 32, 1, dim, 4)
        table = np.array([[2, 0, 3]], np.int32)
        for d0 in range(0, dim, 16):
            q = torch.zeros((1, 16, dim), dtype=torch.float16, device="cuda")
            q[0, torch.arange(16), torch.arange(d0, d0 + 16)] = 8.0
            out, lse = run(api, c, "f16", q, table, [75], 75, scale=1.0)
            check(c, "f16", q, out, lse, table, [75], scale=1.0)


def test_attention_extreme_scores():
    """Large scores of both signs: one position takes everything, or all underflow beside it."""
    api = require_gpu()
    say("attention: extreme scores")
    c = Cache("bf16", "heads", 12, 16, 2, 64, 4)
    table = tables([190], 16, 12, 3)
    q = normal((1, 4, 64), "bf16", 5, sigma=200.0)
    for split in (True, False):
        out, lse = run(api, c, "bf16", q, table, [190], 190, split=split, scale=1.0)
        check(c, "bf16", q, out, lse, table, [190], scale=1.0)
        out, lse = run(api, c, "bf16", q, table, [190], 190, split=split, scale=0.0)
        check(c, "bf16", q, out, lse, table, [190], scale=0.0)


def test_attention_non_finite_values_propagate():
    """A NaN in an attended value spoils its own element of its own head; one in a key spoils the head's rows."""
    api = require_gpu()
    c = Cache("f16", "heads", 12, 16, 2, 64, 4)
    table = tables([190], 16, 12, 3)
    q = normal((1, 4, 64), "f16", 5)
    clean, _ = run(api, c, "f16", q, table, [190], 190)
    j = 77
    c.planes[1][table[0, j // 16], 1, j % 16, 5] = float("nan")
    out, lse = run(api, c, "f16", q, table, [190], 190)
    bad = np.isnan(f64(out))
    assert bad[0, 2:, 5].all() and bad.sum() == 2 and np.isfinite(f64(lse)).all()
    assert np.array_equal(f64(out)[~bad], f64(clean)[~bad])
    c.planes[0][table[0, j // 16], 0, j % 16, 3] = float("nan")
    out, lse = run(api, c, "f16", q, table, [190], 190)
    assert np.isnan(f64(out))[0, :2].all() and np.isnan(f64(lse))[0, :2].all() and np.isfinite(f64(lse))[0, 2:].all()


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_attention_offsets_past_32_bits(cache):
    """Pages past 2^32 bytes of the cache."""
    api = require_gpu()
    say(f"attention {cache}: 4.5 GiB planes")
    page, heads, dim = 64, 4, 128
    size = 1 if cache == "e4m3" else 2
    pages = (9 << 29) // (page * heads * dim * size) + 1
    small = Cache(cache, "heads", 3, page, heads, dim, 6)
    table = np.array([[pages - 1, 1, pages - 3]], np.int32)
    big = []
    for t in small.planes + [s for s in small.scales if s is not None]:
        z = torch.zeros((pages, *t.shape[1:]), dtype=t.dtype, device="cuda")
        z[torch.from_numpy(table[0].astype(np.int64)).cuda()] = t
        big.append(z)
    c = api.KVCache(fmt_of(api, cache), *big)
    q = normal((1, 8, dim), "f16", 5)
    out, lse = torch.empty_like(q), torch.empty((1, 8), device="cuda")
    api.mxattn_decode_run(c, api.MX_F16, q, out, dev(table), dev(np.array([180], np.int32)), 180, dim ** -0.5, lse=lse)
    check(small, "f16", q, out, lse, np.array([[0, 1, 2]], np.int32), [180])


def test_attention_streams_and_graph(monkeypatch):
    """Two streams with a workspace each, and a graph of append and attention replayed between eager calls:
    the bits of the same calls alone."""
    monkeypatch.delenv("MX_SYNC_CHECK", raising=False)
    api = require_gpu()
    say("attention: two streams, graph replays")
    lengths = [4000, 1, 900]
    sets = []
    for i, cache in enumerate(("f16", "e4m3")):
        c = Cache(cache, "heads", 320, 16, 2, 128, i)
        table = tables(lengths, 16, 320, i)
        q = normal((3, 8, 128), "f16", 5 + i)
        sets.append((c, q, dev(table), dev(np.array(lengths, np.int32)), torch.empty_like(q), torch.empty((3, 8), device="cuda"),
                     torch.zeros(api.mxattn_decode_workspace_size(c.c, 3, 8, 4000), dtype=torch.uint8, device="cuda")))

    def call(s, out=None):
        c, q, table, n, o, lse, ws = s
        api.mxattn_decode_run(c.c, api.MX_F16, q, o if out is None else out, table, n, 4000, 0.1, lse=lse, workspace=ws)

    want = []
    for s in sets:
        assert s[6].numel() > 0
        call(s)
        want.append(f64(s[4]))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for s in sets:
        s[4].fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(4):
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                call(s)
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert np.array_equal(f64(s[4]), w)

    c, q, table, n, o, lse, ws = sets[1]
    kv = normal((3, 2, 128), "f16", 77)
    rope = api.Rope(128, dev(np.array(api.mxrope_freqs_host(128, 1e4)[0])))
    pos = dev(np.array([3999, 0, 899], np.int32))
    q2, o2 = torch.empty_like(q), torch.empty_like(q)

    def step(out):
        api.mxkv_append_run(c.c, api.MX_F16, kv, kv, pos, table, rope=rope, q=q, q_out=q2)
        api.mxattn_decode_run(c.c, api.MX_F16, q2, out, table, n, 4000, 0.1, workspace=ws)

    step(o)
    want = f64(o)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(o2)
    for _ in range(3):
        o2.fill_(float("nan"))
        step(o)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(f64(o2), want) and np.array_equal(f64(o), want)


@pytest.mark.parametrize("kind,cache,dim,page", [("f16", "f16", 64, 64), ("bf16", "e4m3", 64, 30), ("f16", "f16", 128, 16)])
def test_attention_joins_many_parts(kind, cache, dim, page):
    """One long row of one head, over every workgroup: its parts are joined in groups first. The same bits every time."""
    api = require_gpu()
    n = 100001
    say(f"attention {cache}: {n} keys of one head of {dim}, pages of {page}")
    pages = -(-n // page) + 1
    c = Cache(cache, "heads", pages, page, 1, dim, 8)
    table = tables([n], page, pages, 3)
    q = normal((1, 5, dim), kind, 5)
    ws = torch.zeros(api.mxattn_decode_workspace_size(c.c, 1, 5, n), dtype=torch.uint8, device="cuda")
    outs = [run(api, c, kind, q, table, [n], n, ws=ws) for _ in range(3)]
    check(c, kind, q, *outs[0], table, [n])
    assert all(torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1]) for o, l in outs[1:])


@pytest.mark.parametrize("window", [0, 700])
def test_attention_many_ragged_rows(window):
    """More rows than lanes, from none to thousands of keys: the shares' cuts fall anywhere."""
    api = require_gpu()
    g = np.random.Generator(np.random.PCG64(12))
    lengths = [int(x) for x in np.exp(g.uniform(0, np.log(4000), 150))]
    lengths[3] = lengths[70] = lengths[149] = 0
    lengths[64] = 4000
    starts = [int(x) for x in g.integers(0, 600, 150)]
    say(f"attention: 150 ragged rows, window={window}")
    pages = sum(-(-n // 32) for n in lengths)
    c = Cache("f16", "slots", pages, 32, 2, 64, 9)
    table = tables(lengths, 32, pages, 3)
    q = normal((150, 4, 64), "f16", 5)
    for s in (None, starts):
        out, lse = run(api, c, "f16", q, table, lengths, 4000, starts=s, window=window)
        check(c, "f16", q, out, lse, table, lengths, s, window)


def test_attention_workspace_serves_other_shapes():
    """One workspace, zero-filled once, for calls of different batches, heads and lengths in turn."""
    api = require_gpu()
    say("attention: one workspace for several shapes")
    sets = []
    for i, (cache, hq, hk, dim, lengths) in enumerate([("f16", 4, 2, 64, [5000]), ("f16", 16, 8, 128, [3000, 10, 900, 1500]),
                                                       ("e4m3", 8, 1, 256, [2000] * 3), ("f16", 96, 12, 32, [700] * 9)]):
        pages = sum(-(-n // 16) for n in lengths)
        c = Cache(cache, "heads", pages, 16, hk, dim, i)
        sets.append((c, normal((len(lengths), hq, dim), "f16", i), tables(lengths, 16, pages, i), lengths))
    need = [api.mxattn_decode_workspace_size(c.c, q.shape[0], q.shape[1], max(n)) for c, q, _, n in sets]
    assert min(need) > 0 and len(set(need)) > 1
    ws = torch.zeros(max(need), dtype=torch.uint8, device="cuda")
    for i in (0, 1, 2, 3, 1, 0, 3, 2, 0):
        c, q, table, lengths = sets[i]
        out, lse = run(api, c, "f16", q, table, lengths, max(lengths), ws=ws)
        check(c, "f16", q, out, lse, table, lengths)


def test_attention_large_bf16_values():
    """Values near bfloat16's largest: the sums of a row stay in range."""
    api = require_gpu()
    say("attention: values of 2^100")
    c = Cache("bf16", "heads", 64, 16, 1, 64, 4)
    c.planes[1] *= 2.0 ** 100
    c.v = c.v * 2.0 ** 100
    table = tables([1000], 16, 64, 3)
    q = normal((1, 4, 64), "bf16", 5)
    for split in (True, False):
        out, lse = run(api, c, "bf16", q, table, [1000], 1000, split=split)
        check(c, "bf16", q, out, lse, table, [1000])


def test_attention_empty_rows_among_many():
    """A batch of empty rows only, with a workspace: zeros and -inf, and the counters stay at zero."""
    api = require_gpu()
    say("attention: empty rows")
    c = Cache("f16", "heads", 40, 16, 2, 128, 4)
    table = tables([0, 600, 0], 16, 40, 3, cols=60)
    q = normal((3, 6, 128), "f16", 5)
    for lengths in ([0, 0, 0], [0, 600, 0], [-1, 600, -2 ** 31]):
        out, lse = run(api, c, "f16", q, table, lengths, 960)
        check(c, "f16", q, out, lse, table, lengths)


@pytest.mark.parametrize("kind,cache,hq,hk,dim,page,seqs,n", [
    ("f16", "f16", 40, 2, 128, 16, 4, 66000), ("bf16", "e4m3", 132, 4, 64, 64, 60, 4400), ("f16", "e4m3", 34, 1, 96, 24, 9, 120000),
    ("bf16", "bf16", 17, 1, 8, 5, 40, 13200), ("f16", "f16", 20, 1, 128, 32, 2400, 250)])
@pytest.mark.parametrize("split", [True, False])
def test_attention_many_heads_to_a_cache_head(kind, cache, hq, hk, dim, page, seqs, n, split):
    """More than 16 query heads per cache head, with enough keys that two tiles of heads meet a key together. Sequences share
    one table row, so that the 64-bit form takes each of their few lengths once."""
    api = require_gpu()
    say(f"attention {cache}: {hq}/{hk} heads of {dim}, {seqs} rows of up to {n}, split={split}")
    if not split and n > 60000:
        seqs = 2
    pages = -(-n // page) + 1
    c = Cache(cache, "heads", pages, page, hk, dim, 8)
    table = np.repeat(tables([n], page, pages, 3), seqs, 0)
    some = [n, n - 129, n // 3, 0, 1]
    lengths = [some[i % 5] if i % 7 == 0 else n for i in range(seqs)]
    q = normal((5, hq, dim), kind, 5)[torch.arange(seqs, device="cuda") % 5]
    out, lse = run(api, c, kind, q, table, lengths, n, split=split)
    firsts = {}
    for i in range(seqs):
        firsts.setdefault((i % 5, lengths[i]), i)
    pick = sorted(firsts.values())[:6]
    check(c, kind, q[pick], out[pick], lse[pick], table[pick], [lengths[i] for i in pick])
    for i in range(seqs):                                   # equal rows, wherever they lie in the batch
        j = firsts[i % 5, lengths[i]]
        tol = 4 * ref.HALF_STEP[kind]
        assert torch.allclose(out[i].float(), out[j].float(), rtol=tol, atol=tol), i


@pytest.mark.parametrize("softcap", [1e6, 1e30, 3e38])
def test_attention_cap_far_above_the_scores(softcap):
    """s^3 / (3 c^2), what such a cap takes off a score of up to 100, is below a half step of it, so the
    bound without a cap holds."""
    api = require_gpu()
    say(f"attention softcap={softcap}")
    c = Cache("bf16", "heads", 12, 16, 2, 64, 4)
    table = tables([190], 16, 12, 3)
    q = normal((1, 4, 64), "bf16", 5, sigma=3.0)
    out, lse = run(api, c, "bf16", q, table, [190], 190, softcap=softcap)
    check(c, "bf16", q, out, lse, table, [190])


@pytest.mark.parametrize("seqs,n", [(64, 2000), (128, 500), (70, 1400)])
def test_attention_rows_of_one_length(seqs, n):
    """Equal rows, whose shares' cuts lie at fractions of a grain: fewer and more sequences than a wave sums up at a
    time, shares of one place to several."""
    api = require_gpu()
    say(f"attention: {seqs} rows of {n}")
    lengths = [n] * seqs
    pages = seqs * (-(-n // 64))
    c = Cache("f16", "heads", pages, 64, 2, 64, 9)
    table = tables(lengths, 64, pages, 3)
    q = normal((seqs, 4, 64), "f16", 5)
    out, lse = run(api, c, "f16", q, table, lengths, n)
    check(c, "f16", q, out, lse, table, lengths)
