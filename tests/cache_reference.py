"""Plain 64-bit forms of the decode step's cache operators (numpy), and the error bounds their kernels
are held to. Written from the formulas in include/mxgemm.h; no code of the library is used."""
import numpy as np

HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # eps / 2 of each type
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}     # half the smallest subnormal
U32 = 2.0 ** -24                                                         # half a step of fp32


def rotate(x, positions, freq, layout, factor=1.0, inverse=False):
    """x [tokens][heads][dim] (float64) with its first 2 len(freq) elements turned; also
    (|a| + |b|) |factor| of every rotated element (0 elsewhere)."""
    x = np.asarray(x, np.float64)
    half = len(freq)
    i = np.arange(half)
    a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
    w = np.multiply.outer(np.asarray(positions, np.longdouble), np.asarray(freq, np.longdouble))
    cos, sin = (np.asarray(f(w), np.float64)[:, None] * factor for f in (np.cos, np.sin))
    if inverse:
        sin = -sin
    out, size = x.copy(), np.zeros_like(x)
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(factor)
    return out, size


def rotate_bound(out, size, kind):
    """The result's rounding, and in fp32: the reduced angle's rounding (at most 1, times pi: 3.2 half
    steps), the sine's (2 ulp: 4), the factor's and its product (2), both products and the sum (3)."""
    return HALF_STEP[kind] * np.abs(out) * (1 + 2.0 ** -8) + 13 * U32 * size + TINY[kind]


def gather(plane, table_row, n, page_size, order):
    """[heads][n][dim] of a plane in float64, and which positions have a page."""
    pages = plane.shape[0]
    j = np.arange(n)
    page = table_row[j // page_size]
    ok = (page >= 0) & (page < pages)
    page = np.where(ok, page, 0)
    rows = plane[page, :, j % page_size] if order == "heads" else plane[page, j % page_size]
    return rows.transpose(1, 0, 2), ok


def attention(q, k, v, scale, softcap=0.0):
    """One row: q [group][dim], k, v [n][dim] in float64 -> out [group][dim], lse [group], the kernel's
    fp32 error on each, and sum p |v| / sum p, which the rounding of the probabilities multiplies."""
    group, dim = q.shape
    n = k.shape[0]
    if n == 0:
        return np.zeros((group, dim)), np.full(group, -np.inf), np.zeros((group, dim)), np.zeros(group), np.zeros((group, dim))
    s = q @ k.T * scale
    size = np.abs(q) @ np.abs(k).T * abs(scale)
    if softcap:
        s = softcap * np.tanh(s / softcap)
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    total = p.sum(-1, keepdims=True)
    out = p @ v / total
    lse = (top + np.log(total))[:, 0]
    # A score's error: its products are exact, its sum takes at most dim additions (a matrix instruction
    # may cut instead of rounding: twice the half step); scale, log2 e and, with a cap, a tanh and two
    # more factors round it; the exponent's difference and the exponential add their own.
    e = (2 * dim * U32 * size).max(-1) + 16 * U32 * (np.abs(s).max(-1) + abs(top[:, 0]) + softcap + 1)
    sums = 2 * (n + 64) * U32                      # the sums over positions and their joining
    spread = p @ np.abs(v) / total
    return out, lse, spread * (2 * e + 2 * sums)[:, None], e + sums + 8 * U32 * (1 + np.abs(lse)), spread

