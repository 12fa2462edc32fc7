"""Rotary positions and the append to a paged cache against 64-bit forms and the host codec."""
import numpy as np
import pytest
import torch

import cache_reference as ref
from cache_common import TORCH, Cache, f64, fmt_of, normal, tables
from gpu_common import dev, host, require_gpu, say

pytestmark = pytest.mark.gpu


def freqs(api, rot, rule="PLAIN", params=()):
    f, factor = api.mxrope_freqs_host(rot, 10000.0, getattr(api, "MXROPE_" + rule), params)
    return np.array(f), factor


def make_rope(api, f, layout, factor=1.0):
    return api.Rope(2 * len(f), dev(f), api.MXROPE_HALF if layout == "half" else api.MXROPE_PAIRS, factor)


def check_rotation(got, x, pos, f, layout, kind, factor, inverse=False):
    want, size = ref.rotate(f64(x), pos, f, layout, float(np.float32(factor)), inverse)
    bound = ref.rotate_bound(want, size, kind)
    rot = 2 * len(f)
    err = np.abs(f64(got) - want)
    assert np.array_equal(f64(got)[..., rot:], f64(x)[..., rot:]), "elements past rot_dim changed"
    worst = (err / bound)[..., :rot].max()
    say(f"worst error / bound {worst:.3f}")
    assert worst <= 1.0


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 1, 8, 2), (1, 32, 128, 128), (3, 5, 80, 32), (33, 7, 96, 96), (700, 3, 64, 48),
                                                  (2, 65, 256, 256), (5, 4, 72, 20), (1, 200, 128, 64), (2500, 2, 40, 40), (4, 1, 256, 254),
                                                  (300, 17, 248, 2)])
def test_rotary(kind, layout, tokens, heads, dim, rot):
    api = require_gpu()
    say(f"rotary {kind} {layout} tokens={tokens} heads={heads} dim={dim} rot={rot}")
    f, factor = freqs(api, rot, "YARN", (16.0, 4096.0, 32.0, 1.0))
    r = make_rope(api, f, layout, factor)
    x = normal((tokens, heads + 3, dim + 8), kind, 7)[:, 1:heads + 1, 8:]        # strides of its own
    pos = np.random.Generator(np.random.PCG64(3)).integers(-5, 1 << 20, tokens).astype(np.int32)
    pos[0] = (1 << 20) - 1
    p = dev(pos)
    for inverse in (False, True):
        room = torch.full((tokens, heads, dim + 16), 5.0, dtype=x.dtype, device="cuda")
        out = room[..., :dim]
        api.mxrope_run(fmt_of(api, kind), r, x, out, p, inverse=inverse)
        check_rotation(out, x, pos, f, layout, kind, factor, inverse)
        assert bool((room[..., dim:] == 5.0).all()), "written past a row's end"
        same = x.clone()
        api.mxrope_run(fmt_of(api, kind), r, same, same, p, inverse=inverse)     # in place: the same bits
        assert torch.equal(same, out)


def test_rotary_far_positions_and_zero():
    api = require_gpu()
    f, _ = freqs(api, 128)
    r = make_rope(api, f, "half")
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1], np.int32)
    x = normal((6, 2, 128), "f32", 11)
    out = torch.empty_like(x)
    say("rotary: positions up to 2^31")
    api.mxrope_run(api.MX_F32, r, x, out, dev(pos))
    assert torch.equal(out[0], x[0])
    check_rotation(out, x, pos, f, "half", "f32", 1.0)


def test_rotary_gradient_by_differences():
    """The inverse call is the forward's transpose: d(sum w y) / dx by central differences in 64 bits."""
    api = require_gpu()
    g = np.random.Generator(np.random.PCG64(5))
    f, factor = freqs(api, 20, "YARN", (4.0, 512.0, 32.0, 1.0))
    for layout in ("half", "pairs"):
        say(f"rotary gradient {layout}")
        x, w = g.standard_normal((2, 3, 24)), normal((2, 3, 24), "f32", 9)
        pos = np.array([3, 4000], np.int32)
        grad = torch.empty_like(w)
        api.mxrope_run(api.MX_F32, make_rope(api, f, layout, factor), w, grad, dev(pos), inverse=True)
        num, h = np.zeros_like(x), 1e-3
        for i in np.ndindex(x.shape):
            d = np.zeros_like(x)
            d[i] = h
            up, down = (ref.rotate(x + s * d, pos, f, layout, float(np.float32(factor)))[0] for s in (1, -1))
            num[i] = ((up - down) * f64(w)).sum() / (2 * h)
        # the form is linear: differences in 64 bits are good to 2^-40 here, the kernel to rotate_bound's 13 half steps
        assert np.abs(f64(grad) - num).max() <= 16 * ref.U32 * 2 * np.abs(f64(w)).max() * factor


def test_rotary_non_finite_stay_in_their_pair():
    api = require_gpu()
    f, _ = freqs(api, 32)
    for layout, partner in (("half", lambda i: i + 16), ("pairs", lambda i: i + 1)):
        x = normal((1, 1, 40), "f16", 2)
        x[0, 0, 4], x[0, 0, 37] = float("inf"), float("nan")
        out = torch.empty_like(x)
        api.mxrope_run(api.MX_F16, make_rope(api, f, layout), x, out, dev(np.array([7], np.int32)))
        bad = set(np.flatnonzero(~np.isfinite(f64(out)[0, 0])))
        assert bad == {4, partner(4), 37}


# ---- append --------------------------------------------------------------------------------------

APPENDS = [  # tokens, seqs, q heads, heads, dim, page, rot, layout
    (1, 1, 4, 1, 32, 1, 32, "half"), (5, 5, 32, 8, 128, 16, 128, "half"), (37, 3, 6, 3, 96, 24, 40, "pairs"),
    (64, 64, 8, 8, 64, 64, 64, "pairs"), (300, 2, 7, 7, 256, 5, 20, "half"), (2100, 4, 2, 2, 160, 32, 160, "half"),
    (9, 2, 40, 40, 224, 16, 0, "half")]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("order", ["heads", "slots"])
@pytest.mark.parametrize("tokens,seqs,hq,hk,dim,page,rot,layout", APPENDS)
def test_append(kind, quant, order, tokens, seqs, hq, hk, dim, page, rot, layout):
    """Slots of tokens hold the rotated keys (the bits of mxrope_run, quantised as the host codec does) and
    the values; every other slot keeps what it held."""
    api = require_gpu()
    say(f"append {kind} quant={quant} {order} tokens={tokens} heads={hq}/{hk} dim={dim} page={page} rot={rot}")
    g = np.random.Generator(np.random.PCG64(tokens + dim))
    seq = np.sort(g.integers(0, seqs, tokens)).astype(np.int32)
    first = g.integers(0, 200, seqs)
    pos = np.array([first[s] + np.sum(seq[:t] == s) for t, s in enumerate(seq)], np.int32)
    lengths = [int(first[s] + np.sum(seq == s)) for s in range(seqs)]
    pages = sum(-(-n // page) for n in lengths) + 2
    table = tables(lengths, page, pages, 4)
    c = Cache("e4m3" if quant else kind, order, pages, page, hk, dim, 5)
    before = [t.clone() for t in c.planes + [s for s in c.scales if s is not None]]
    qkv = normal((tokens, hq + 2 * hk, dim), kind, 6)
    qkv[0, hq, :32] = 0.0                                       # a block of zeros
    if tokens > 3:
        qkv[3, hq, 5], qkv[3, hq + hk, 7] = float("inf"), float("nan")
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    fmt, p = fmt_of(api, kind), dev(pos)
    rope, q_out, turned = None, None, k
    if rot:
        f, factor = freqs(api, rot, "NTK", (8.0,))
        rope = make_rope(api, f, layout, factor)
        q_out, turned, want_q = torch.zeros_like(q.contiguous()), torch.empty_like(k.contiguous()), torch.empty_like(q.contiguous())
        api.mxrope_run(fmt, rope, k, turned, p)
        api.mxrope_run(fmt, rope, q, want_q, p)
    api.mxkv_append_run(c.c, fmt, k, v, p, dev(table), seq=dev(seq), rope=rope, q=q if rot else None, q_out=q_out)
    if rot:
        assert torch.equal(q_out, want_q)
    page_of, slot = table[seq, pos // page].astype(np.int64), (pos % page).astype(np.int64)
    want = [t.clone().cpu() for t in before]
    for i, x in enumerate((turned, v)):
        if quant:
            x32 = np.ascontiguousarray(x.float().cpu().numpy())
            codes, scales = np.zeros(x32.shape, np.uint8), np.zeros((*x32.shape[:2], dim // 32), np.uint8)
            api.mx_pack_host(api.MX_E4M3, x32, tokens * hk, dim, codes, scales)
            c.rows(want[i])[page_of, slot] = torch.from_numpy(codes)
            c.rows(want[2 + i])[page_of, slot] = torch.from_numpy(scales)
        else:
            c.rows(want[i])[page_of, slot] = x.cpu()
    torch.cuda.synchronize()
    for got, w in zip(c.planes + [s for s in c.scales if s is not None], want):
        a, b = (t.cpu().contiguous().view(torch.uint8 if quant else torch.int16) for t in (got, w))
        assert torch.equal(a, b)


def test_append_drops_tokens_without_a_slot():
    """Bad sequences, positions and pages: nothing is written for them, their queries are still turned, and
    tokens beside them are written."""
    api = require_gpu()
    say("append: tokens out of range")
    c = Cache("f16", "heads", 4, 8, 2, 32, 1, fill=3.0)
    table = np.array([[0, -1, 4], [2, 3, 1 << 30]], np.int32)
    seq = np.array([0, 0, 0, 1, 1, 1, -1, 2, 1], np.int32)
    pos = np.array([1, 8, 16, -1, 9, 16, 0, 0, 24], np.int32)            # kept: tokens 0 and 4
    k, v, q = (normal((9, n, 32), "f16", n + s) for n, s in ((2, 0), (2, 10), (4, 0)))
    q_out, want = torch.zeros_like(q), torch.zeros_like(q)
    rope = make_rope(api, freqs(api, 32)[0], "half")
    api.mxkv_append_run(c.c, api.MX_F16, k, v, dev(pos), dev(table), seq=dev(seq), rope=rope, q=q, q_out=q_out)
    api.mxrope_run(api.MX_F16, rope, q, want, dev(pos))
    assert torch.equal(q_out, want)
    vals = c.planes[1].cpu().clone()
    assert torch.equal(vals[0, :, 1], v[0].cpu()) and torch.equal(vals[3, :, 1], v[4].cpu())
    vals[0, :, 1] = vals[3, :, 1] = 3.0
    assert bool((vals == 3.0).all())
    assert int((c.planes[0] != 3.0).any(-1).sum()) == 4                   # two tokens of two heads
    api.mxkv_append_run(c.c, api.MX_F16, k[:0], v[:0], dev(pos[:0]), dev(table))   # no token: nothing


def test_append_queries_in_place_and_without_seq():
    api = require_gpu()
    c = Cache("bf16", "slots", 6, 16, 2, 64, 1)
    k, v, q = (normal((3, n, 64), "bf16", n) for n in (2, 2, 6))
    pos, table = dev(np.array([0, 15, 3], np.int32)), dev(np.array([[5], [0], [2]], np.int32))
    rope = make_rope(api, freqs(api, 64)[0], "pairs")
    want = torch.empty_like(q)
    api.mxrope_run(api.MX_BF16, rope, q, want, pos)
    api.mxkv_append_run(c.c, api.MX_BF16, k, v, pos, table, rope=rope, q=q, q_out=q)
    assert torch.equal(q, want)
    assert torch.equal(c.planes[1][5, 0], v[0]) and torch.equal(c.planes[1][0, 15], v[1]) and torch.equal(c.planes[1][2, 3], v[2])


def test_append_offsets_past_32_bits():
    """A cache whose last page starts past 2^32 bytes (and 2^31 elements)."""
    api = require_gpu()
    say("append: 4.5 GiB cache")
    page, heads, dim = 64, 8, 128
    pages = (9 << 29) // (page * heads * dim * 2) + 1
    store = torch.zeros((pages, heads, page, dim), dtype=torch.float16, device="cuda")
    c = api.KVCache(api.MX_F16, store, store)
    k = normal((1, heads, dim), "f16", 1)
    api.mxkv_append_run(c, api.MX_F16, k, k, dev(np.array([63], np.int32)), dev(np.array([[pages - 1]], np.int32)))
    assert torch.equal(store[-1, :, 63], k[0])
    store[-1, :, 63] = 0
    assert not bool(store[-2:].any()) and not bool(store[:2].any())
