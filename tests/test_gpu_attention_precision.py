"""Attention of one new token keeps its probabilities to more than 16 bits: the formula in 64 bits under a bound that
has no rounding of them, only the result's."""
import numpy as np
import pytest
import torch

import cache_reference as ref
from cache_common import Cache, f64, fmt_of, normal, tables
from gpu_common import dev, require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("cache,hq,dim,page,n,sigma", [
    ("same", 4, 8, 16, 2, 1.0), ("same", 32, 32, 16, 3, 1.0), ("same", 16, 32, 5, 30, 1.0), ("e4m3", 16, 32, 16, 30, 1.0),
    ("same", 16, 64, 16, 700, 1.0), ("e4m3", 20, 64, 24, 1000, 1.0), ("same", 16, 136, 16, 700, 1.0), ("same", 40, 64, 16, 33000, 6.0)])
def test_probabilities_are_not_rounded_to_16_bits(kind, cache, hq, dim, page, n, sigma):
    """Each probability is held as its 16-bit value, cut off, and the 16-bit value of what that leaves (below 2 HALF_STEP of it),
    which leaves 2 HALF_STEP^2 of it, or, where binary16 ends (the largest is 2^15), 2^-39 of the largest. In long rows each element has a value at two
    positions only, so that roundings do not average out."""
    api = require_gpu()
    seqs = 4 if n > 10000 else 2                     # enough keys for two tiles of heads to meet a key together
    say(f"attention {kind} over {cache}: {hq} heads of {dim}, {n} keys, pages of {page}")
    pages = -(-n // page) + 1
    c = Cache(kind if cache == "same" else cache, "heads", pages, page, 1, dim, 21)
    table = np.repeat(tables([n], page, pages, 3), seqs, 0)
    if n >= 700:
        g = np.random.Generator(np.random.PCG64(2))
        none = np.ones((pages, 1, page, dim), bool)
        for d in range(dim):
            j = g.integers(0, n, 2)
            none[table[0, j // page], 0, j % page, d] = False
        c.planes[1][torch.from_numpy(none).cuda()] = 0
        c.v = np.where(none, 0.0, c.v)
    q = normal((seqs, hq, dim), kind, 5, sigma)
    need = api.mxattn_decode_workspace_size(c.c, seqs, hq, n)
    ws = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")
    out, lengths = torch.empty_like(q), dev(np.full(seqs, n, np.int32))
    api.mxattn_decode_run(c.c, fmt_of(api, kind), q, out, dev(table), lengths, n, dim ** -0.5, workspace=ws)
    k, _ = ref.gather(c.k, table[0], n, page, "heads")
    v, _ = ref.gather(c.v, table[0], n, page, "heads")
    half = ref.HALF_STEP[kind]
    worst = 0.0
    for b in range(seqs):
        want, _, eo, _, spread = ref.attention(f64(q)[b], k[0], v[0], float(np.float32(dim ** -0.5)))
        bound = eo + half * np.abs(want) * (1 + 2.0 ** -6) + 2 * half ** 2 * spread * (1 + 2.0 ** -6) + n * 2.0 ** -39 * np.abs(v).max() + ref.TINY[kind]
        worst = max(worst, (np.abs(f64(out)[b] - want) / bound).max())
    say(f"worst error / bound {worst:.3f}")
    assert worst <= 1.0


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim,page,n", [(64, 16, 40), (64, 5, 40), (128, 16, 3000), (128, 24, 3000), (256, 16, 3000)])
def test_infinite_values_stay_infinite(kind, dim, page, n):
    """An infinite value among finite ones, or several of one sign, make their element that infinity; of both signs NaN; all
    beside them stays as it was. Scores of 0 (every probability is a power of two) and others."""
    api = require_gpu()
    say(f"attention {kind}: infinite values, {n} keys of {dim}, pages of {page}")
    pages = -(-n // page)
    c = Cache(kind, "slots", pages, page, 2, dim, 21)
    table = tables([n], page, pages, 3)
    ws = torch.zeros(max(16, api.mxattn_decode_workspace_size(c.c, 1, 8, n)), dtype=torch.uint8, device="cuda")
    lengths, t = dev(np.array([n], np.int32)), dev(table)
    for sigma in (0.0, 1.0):
        q = normal((1, 8, dim), kind, 5, sigma)

        def run(plane):
            out = torch.empty_like(q)
            api.mxattn_decode_run(api.KVCache(fmt_of(api, kind), c.planes[0], plane, order=api.MXKV_SLOTS_FIRST), fmt_of(api, kind), q, out, t, lengths, n,
                                  dim ** -0.5, workspace=ws)
            return f64(out)[0]

        plane = c.planes[1].clone()
        clean = run(plane)

        def put(j, d, x):
            plane[int(table[0, j // page]), j % page, 1, d] = x

        put(7, 3, float("inf")), put(n - 1, 5, float("-inf")), put(0, 8, float("inf")), put(n // 2, 8, float("inf"))
        put(1, 9, float("inf")), put(n - 2, 9, float("-inf"))
        got = run(plane)
        assert np.all(got[4:, 3] == np.inf) and np.all(got[4:, 5] == -np.inf) and np.all(got[4:, 8] == np.inf) and np.isnan(got[4:, 9]).all()
        same = np.ones((8, dim), bool)
        same[4:, [3, 5, 8, 9]] = False
        assert np.array_equal(got[same], clean[same])


@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("page,n", [(16, 200), (24, 200), (16, 2000), (24, 2000)])
def test_nan_keys_spoil_their_head(kind, cache, page, n):
    """A NaN in an attended key makes its head's rows and lse NaN, cut to 16 bits or not, and no others."""
    api = require_gpu()
    say(f"attention {kind} over {cache}: a NaN key among {n}, pages of {page}")
    pages = -(-n // page)
    c = Cache(cache, "heads", pages, page, 2, 64, 21)
    table = tables([n], page, pages, 3)
    ws = torch.zeros(max(16, api.mxattn_decode_workspace_size(c.c, 1, 8, n)), dtype=torch.uint8, device="cuda")
    q = normal((1, 8, 64), kind, 5)
    for j in (0, n // 2, n - 1):
        place = (int(table[0, j // page]), 1, j % page, 9)
        old = c.planes[0][place].clone()
        c.planes[0][place] = 0x7F if cache == "e4m3" else float("nan")
        out, lse = torch.zeros_like(q), torch.zeros(1, 8, device="cuda")
        api.mxattn_decode_run(c.c, fmt_of(api, kind), q, out, dev(table), dev(np.array([n], np.int32)), n, 0.125, lse=lse, workspace=ws)
        c.planes[0][place] = old
        assert np.isnan(f64(out)[0, 4:]).all() and np.isnan(f64(lse)[0, 4:]).all() and np.isfinite(f64(out)[0, :4]).all() and np.isfinite(f64(lse)[0, :4]).all(), j
