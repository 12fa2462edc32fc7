"""RMS norm with weights far from 1: products of an element and its weight that leave fp32's range, where the result does not."""
import numpy as np
import pytest
import torch

from cache_common import TORCH, f64, fmt_of
from cache_reference import HALF_STEP, TINY, U32
from gpu_common import host, require_gpu, say
from test_gpu_norm import reference, relative, rows_of

pytestmark = pytest.mark.gpu

# powers of two of a row's elements and of the weights: both large, both small, each with each
FAR = [(15, 118), (60, 100), (100, 20), (62, 118), (-15, -110), (-40, -100), (-45, -84), (-100, -30), (-60, 100), (60, -100), (0, 118), (0, -110)]
EIGHT = {"MX_E4M3": (3, 8, 448.0, -9, torch.float8_e4m3fn), "MX_E5M2": (2, 15, 57344.0, -16, torch.float8_e5m2)}


def inputs(kind, dim, a, b, seed):
    """Normal elements of size 2^a and weights of size 2^b; the second row is zeros but for one element, the third zeros."""
    g = torch.Generator().manual_seed(seed)
    x, w = torch.randn(3, dim, generator=g, dtype=torch.float64), torch.randn(dim, generator=g, dtype=torch.float64)
    x[1, :dim // 2], x[1, dim // 2 + 1:], x[2] = 0, 0, 0
    return rows_of((x * 2.0 ** a).to(TORCH[kind]).cuda()), (w * 2.0 ** b).to(TORCH[kind]).cuda()


def eps_of(a):
    """2^-20 of the rows' mean square, as far as fp32 goes."""
    return float(np.float32(2.0 ** (2 * min(max(a, -60), 60) - 20)))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [24, 4128, 40000])
@pytest.mark.parametrize("a,b", FAR)
def test_same_type(kind, dim, a, b):
    api = require_gpu()
    x, w = inputs(kind, dim, a, b, 1)
    eps = eps_of(a)
    out = rows_of(torch.zeros_like(x))
    api.mxnorm_run(fmt_of(api, kind), x, out, None, fmt_of(api, kind), weight=w, eps=eps)
    _, y = reference(x, None, w, eps)
    got = f64(out)
    assert np.isfinite(got).all() and not got[2].any()
    # an element 2^-126 below the row's size may lose its last bits before the weight multiplies it
    bound = np.abs(y) * (HALF_STEP[kind] * 1.01 + relative(dim) + U32) + TINY[kind] + 2.0 ** -149 * np.abs(f64(w))
    err = np.abs(got - y) / bound
    say(f"{kind} {dim} elements 2^{a} weights 2^{b}: worst error / bound {err.max():.3f}")
    assert err.max() <= 1.0


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [24, 4128, 40000])
@pytest.mark.parametrize("a,b", FAR)
def test_int8(kind, dim, a, b):
    api = require_gpu()
    x, w = inputs(kind, dim, a, b, 2)
    eps = eps_of(a)
    q, s = rows_of(torch.full(x.shape, 7, dtype=torch.int8, device="cuda")), torch.full((3,), 7.0, device="cuda")
    api.mxnorm_run(fmt_of(api, kind), x, q, s, api.MX_INT8, weight=w, eps=eps)
    _, y = reference(x, None, w, eps)
    q, s, most = f64(q), f64(s), np.abs(y).max(-1)
    assert s[2] == 0 and not q[2].any()
    assert np.all(np.abs(s - most / 127) <= most / 127 * (relative(dim) + 6 * U32) + TINY["f32"])
    err = np.abs(q[:2] - 127 * y[:2] / most[:2, None]).max()
    say(f"{kind} {dim} elements 2^{a} weights 2^{b}: worst {err:.5f} steps")
    assert err <= 0.5 + 127 * (relative(dim) + 6 * U32)


@pytest.mark.parametrize("fmt", ["MX_E4M3", "MX_E5M2"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [32, 4128, 40000])
@pytest.mark.parametrize("a,b", FAR)
def test_blocks(fmt, kind, dim, a, b):
    api = require_gpu()
    bits, top, most, least, kind8 = EIGHT[fmt]
    x, w = inputs(kind, dim, a, b, 3)
    eps = eps_of(a)
    codes, scales = torch.full(x.shape, 0x5A, dtype=torch.uint8, device="cuda"), torch.full((3, dim // 32), 0x5A, dtype=torch.uint8, device="cuda")
    api.mxnorm_run(fmt_of(api, kind), x, codes, scales, getattr(api, fmt), weight=w, eps=eps)
    _, y = reference(x, None, w, eps)
    assert not bool((codes[2] & 0x7F).any()) and not bool(scales[2].any())  # zeros, of their weights' signs
    rel = relative(dim)
    amax, e = np.abs(y).reshape(3, -1, 32).max(-1), host(scales).astype(int) - 127
    with np.errstate(divide="ignore"):
        lo, hi = (np.maximum(np.floor(np.log2(amax * (1 + s * rel))) - top, -127) for s in (-1, 1))
    assert np.all((e == lo) | (e == hi))
    step = np.repeat(2.0 ** e, 32, axis=1)
    got, want = f64(codes.view(kind8)) * step, np.clip(y, -most * step, most * step)
    # elements that fp32 holds in fewer bits: half of its smallest step too
    bound = np.maximum(np.abs(y) * 2.0 ** -(bits + 1), 2.0 ** (least - 1) * step) * (1 + 4 * rel) + np.abs(y) * rel + TINY["f32"]
    err = (np.abs(got - want) / bound).max()
    say(f"{fmt} {kind} {dim} elements 2^{a} weights 2^{b}: worst error / bound {err:.3f}")
    assert err <= 1.0


@pytest.mark.parametrize("fmt", ["MX_E4M3", "MX_F32", "MX_INT8"])
def test_infinite_weight(fmt):
    """A weight that is infinite or NaN reaches its own column, or the blocks and integer rows that it is in."""
    api = require_gpu()
    dim = 4096
    for bad in (float("inf"), float("nan")):
        x, w = inputs("f32", dim, 0, 0, 4)
        w[70] = bad
        if fmt == "MX_F32":
            out = torch.zeros_like(x)
            api.mxnorm_run(api.MX_F32, x, out, None, api.MX_F32, weight=w, eps=1e-6)
            fine = torch.isfinite(out)
            assert not bool(fine[0, 70]) and int((~fine[0]).sum()) == 1
        elif fmt == "MX_INT8":
            q, s = torch.full((3, dim), 7, dtype=torch.int8, device="cuda"), torch.zeros(3, device="cuda")
            api.mxnorm_run(api.MX_F32, x, q, s, api.MX_INT8, weight=w, eps=1e-6)
            assert bool(s.isnan().all()) and not bool(q.any())
        else:
            codes, scales = torch.full((3, dim), 7, dtype=torch.uint8, device="cuda"), torch.zeros(3, dim // 32, dtype=torch.uint8, device="cuda")
            api.mxnorm_run(api.MX_F32, x, codes, scales, api.MX_E4M3, weight=w, eps=1e-6)
            assert int((scales[0] == 255).sum()) == 1 and scales[0, 2].item() == 255 and not bool(codes[0, 64:96].any())
