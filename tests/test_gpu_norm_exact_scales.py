"""Scales of blocks whose largest element is at a power of two: rows of elements of one size, whose norm is known without any rounding."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from cache_common import TORCH, f64, fmt_of
from gpu_common import host, require_gpu, say

pytestmark = pytest.mark.gpu
COUNT = 200  # rows, each of its own constant
# Elements within this of a power of two, relative to it, count as the power: 64 bits lose at most (dim / 64 + 30) 2^-53 of the sum, half of it in the root.
NEAR = Fraction(1, 2 ** 40)


def constants(kind, seed):
    """Numbers in [1, 2) of random mantissas, exact in `kind`."""
    bits = {"f16": 10, "bf16": 7, "f32": 23}[kind]
    g = np.random.Generator(np.random.PCG64(seed))
    return 1.0 + g.integers(0, 2 ** bits, COUNT) / 2.0 ** bits


@pytest.mark.parametrize("fmt,top", [("MX_E4M3", 8), ("MX_E5M2", 15)])
@pytest.mark.parametrize("dim", [32, 64, 96, 1024, 4096, 8192, 40000])
@pytest.mark.parametrize("kind,eps,size", [(k, *x) for k in ("f16", "bf16", "f32") for x in ((0.0, 0), (2.0 ** -36, 0), (2.0 ** -30, 3))] +
                         [(k, 0.0, size) for k in ("bf16", "f32") for size in (60, -80)])
def test_rows_of_one_size(fmt, top, kind, dim, eps, size):
    """Rows of +-c have y = +-c / sqrt(c^2 + eps): exactly 1 without eps, below 1 by eps / (2 c^2), less than fp32 shows, with a small one."""
    api = require_gpu()
    c = constants(kind, dim) * 2.0 ** size
    sign = np.where(np.arange(dim) % 3 == 0, -1.0, 1.0)
    x = torch.from_numpy(c[:, None] * sign).to(TORCH[kind]).cuda()
    assert np.array_equal(f64(x)[:, 1], c)
    codes, scales = torch.zeros(COUNT, dim, dtype=torch.uint8, device="cuda"), torch.zeros(COUNT, dim // 32, dtype=torch.uint8, device="cuda")
    api.mxnorm_run(fmt_of(api, kind), x, codes, scales, getattr(api, fmt), eps=eps)
    # y < 1 - 2^-40 means eps above 2^-39 of c^2
    below = np.array([Fraction(eps) > 2 * NEAR * Fraction(float(v)) ** 2 for v in c])
    want = 127 - top - below.astype(int)
    got = host(scales).astype(int)
    say(f"{fmt} {kind} {dim} eps {eps}: {int((got != want[:, None]).any(1).sum())} of {COUNT} rows differ")
    assert np.array_equal(got, np.broadcast_to(want[:, None], got.shape))


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 2048, 40000])
def test_weights_take_elements_to_powers_of_two(kind, dim):
    """y = w for rows of one size: weights that are powers of two, one step below them and one above, each alone at its block's top."""
    api = require_gpu()
    step = {"f16": 2.0 ** -10, "bf16": 2.0 ** -7, "f32": 2.0 ** -23}[kind]
    x = torch.from_numpy(np.repeat(constants(kind, 5)[:, None], dim, 1)).to(TORCH[kind]).cuda()
    w = np.full(dim, 0.25)
    at = np.arange(dim // 32)
    power = 2.0 ** (at % 7)
    w[32 * at + at % 32] = power * np.array([1.0, 1.0 - step / 2, 1.0 + step])[at % 3]
    weight = torch.from_numpy(w).to(TORCH[kind]).cuda()
    assert np.array_equal(f64(weight), w)
    codes, scales = torch.zeros(COUNT, dim, dtype=torch.uint8, device="cuda"), torch.zeros(COUNT, dim // 32, dtype=torch.uint8, device="cuda")
    api.mxnorm_run(fmt_of(api, kind), x, codes, scales, api.MX_E4M3, weight=weight, eps=0.0)
    want = np.floor(np.log2(w.reshape(-1, 32).max(1))).astype(int) - 8 + 127
    got = host(scales).astype(int)
    assert np.array_equal(got, np.broadcast_to(want, got.shape)), (got != want).any(1).sum()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_longest_rows(kind):
    """Rows of 2^20 elements, whose sums lose the most: exactly 1, and below it by 2^-38 and more."""
    api = require_gpu()
    dim, c = 1 << 20, constants(kind, 9)[:4]
    x = torch.from_numpy(np.repeat(c[:, None], dim, 1)).to(TORCH[kind]).cuda()
    codes, scales = torch.zeros(4, dim, dtype=torch.uint8, device="cuda"), torch.zeros(4, dim // 32, dtype=torch.uint8, device="cuda")
    for eps, below in ((0.0, 0), (2.0 ** -35, 1)):
        api.mxnorm_run(fmt_of(api, kind), x, codes, scales, api.MX_E4M3, eps=eps)
        assert bool((scales == 119 - below).all()), eps
