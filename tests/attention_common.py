"""Shared by the GPU tests of attention over rows that are cut into shares: one call with its workspace, whose counters have to be
back at zero, and the comparison with the formula in 64 bits."""
import numpy as np
import torch

import cache_reference as ref
from cache_common import f64, fmt_of
from gpu_common import dev, require_gpu, say

COUNTERS = 3 * 512 * 4   # bytes of the counters at a workspace's beginning: three for each workgroup of the largest grid


def workspace(c, seqs, hq, max_len, window=0):
    """A zero-filled workspace of the size asked for, which has to be one: rows of these sizes are cut."""
    need = require_gpu().mxattn_decode_workspace_size(c.c, seqs, hq, max_len, window)
    assert need > COUNTERS, "rows of these sizes are not cut"
    return torch.zeros(need, dtype=torch.uint8, device="cuda")


def attend(c, kind, q, table, lengths, max_len, ws=None, starts=None, window=0, softcap=0.0, scale=None):
    api = require_gpu()
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 99.0, device="cuda")
    api.mxattn_decode_run(c.c, fmt_of(api, kind), q, out, dev(table), dev(np.asarray(lengths, np.int32)), max_len,
                          q.shape[2] ** -0.5 if scale is None else scale, lse=lse, starts=None if starts is None else dev(np.asarray(starts, np.int32)),
                          window=window, softcap=softcap, workspace=ws)
    if ws is not None:
        torch.cuda.synchronize()
        assert not bool(ws[:COUNTERS].any()), "counters not back at zero"
    return out, lse


def check(c, kind, q, out, lse, table, lengths, starts=None, window=0, softcap=0.0, scale=None):
    """Every row against the formula: the bound counts the kernel's fp32 steps, the two 16-bit values that hold a probability (2 HALF_STEP^2
    of it is left, or 2^-39 of the largest in binary16) and the result's rounding."""
    q64, o64, l64 = f64(q), f64(out), f64(lse)
    n, hq, dim = q64.shape
    share, half = hq // c.heads, ref.HALF_STEP[kind]
    scale = float(np.float32(dim ** -0.5 if scale is None else scale))
    worst = [0.0, 0.0]
    for b in range(n):
        hi = max(0, min(int(lengths[b]), table.shape[1] * c.page))
        lo = max(0, int(starts[b])) if starts is not None else 0
        lo = max(lo, hi - window) if window else lo
        k, ok = ref.gather(c.k, table[b], hi, c.page, c.order)
        v, _ = ref.gather(c.v, table[b], hi, c.page, c.order)
        ok &= np.arange(hi) >= lo
        for h in range(c.heads):
            at = slice(h * share, (h + 1) * share)
            if not ok.any():
                assert not o64[b, at].any() and np.all(l64[b, at] == -np.inf), (b, h)
                continue
            vals = v[h][ok]
            want, wl, eo, el, spread = ref.attention(q64[b, at], k[h][ok], vals, scale, softcap)
            bound = eo + (half * np.abs(want) + 2 * half ** 2 * spread) * (1 + 2.0 ** -6) + len(vals) * 2.0 ** -39 * np.abs(vals).max() + ref.TINY[kind]
            assert np.all(np.isfinite(o64[b, at])), (b, h)
            worst = [max(worst[0], (np.abs(o64[b, at] - want) / bound).max()), max(worst[1], (np.abs(l64[b, at] - wl) / el).max())]
    say(f"worst error / bound: out {worst[0]:.3f}, lse {worst[1]:.3f}")
    assert worst[0] <= 1.0 and worst[1] <= 1.0, worst


def hide(c, table, lengths, starts=None, window=0):
    """NaN in every slot that no row attends."""
    seen = np.zeros((c.planes[0].shape[0], c.page), bool)
    for b, n in enumerate(lengths):
        j = np.arange(max(0, n))
        lo = max(0, int(starts[b])) if starts is not None else 0
        j = j[j >= (max(lo, n - window) if window else lo)]
        p = table[b][j // c.page]
        ok = (p >= 0) & (p < len(seen))
        seen[p[ok], j[ok] % c.page] = True
    dead = torch.from_numpy(~seen).cuda()
    for plane, scale in zip(c.planes, c.scales):
        if scale is not None:
            c.rows(plane)[dead], c.rows(scale)[dead] = 0x7F, 0xFF
        else:
            c.rows(plane)[dead] = float("nan")
