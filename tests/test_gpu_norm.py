"""RMS norm with the residual's addition and the quantisation of rows, against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

from cache_common import TORCH, f64, fmt_of, normal
from cache_reference import HALF_STEP, TINY, U32
from gpu_common import dev, host, require_gpu, say

pytestmark = pytest.mark.gpu

# (rows, dim): single elements, tails, each kernel shape's first and last width, rows that are read twice
SHAPES = [(1, 1), (3, 7), (2, 8), (5, 33), (1, 1024), (6, 1025), (1, 4096), (70, 1000), (1030, 1032), (1030, 4096), (3, 4104), (1027, 4104),
          (2, 16384), (1026, 16384), (2, 16392), (1, 32768), (2, 32776), (1, 100003)]


def rows_of(x, pad=0):
    """The same values in rows of whole 16-byte pieces, `pad` pieces more, the rest filled with NaN or 0x5A."""
    unit = 16 // x.element_size()
    wide = -(-x.shape[1] // unit) * unit + pad * unit
    y = torch.full((x.shape[0], wide), float("nan") if x.is_floating_point() else 0x5A, dtype=x.dtype, device="cuda")
    y[:, :x.shape[1]] = x
    return y[:, :x.shape[1]]


def relative(dim):
    """Of y in fp32: the sum of squares (a thread's terms one by one, then the lanes' and waves') and its root, rsqrt (an ulp), eps and the
    mean, two products."""
    return ((dim / 64 + 24) / 2 + 2 + 2 + 3) * U32


def reference(x, residual, weight, eps):
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    z = f64(h)
    y = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps)
    return h, y if weight is None else y * f64(weight)


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_norm_same_type(kind, rows, dim):
    api = require_gpu()
    x, w = rows_of(normal((rows, dim), kind, 1), rows % 2), normal((dim,), kind, 2)
    out = rows_of(torch.zeros(rows, dim, dtype=TORCH[kind], device="cuda"), 1)
    api.mxnorm_run(fmt_of(api, kind), x, out, None, fmt_of(api, kind), weight=w, eps=1e-6)
    _, y = reference(x, None, w, float(np.float32(1e-6)))
    err = np.abs(f64(out) - y) / (np.abs(y) * (HALF_STEP[kind] * 1.01 + relative(dim)) + TINY[kind])
    say(f"norm {kind} {rows}x{dim}: worst error / bound {err.max():.3f}")
    assert err.max() <= 1.0
    if out.stride(0) > dim:  # what is between the rows stays
        assert bool(torch.as_strided(out, (rows, out.stride(0) - dim), (out.stride(0), 1), dim).isnan().all())


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,dim,where", [(1, 5, "new"), (7, 96, "x"), (1030, 640, "residual"), (1026, 2048, "new"), (4, 4096, "residual"), (2, 5003, "x"),
                                            (1030, 9000, "x"), (2, 50000, "residual"), (3, 40008, None)])
def test_norm_residual_int8(kind, rows, dim, where):
    """The sum is exact in its rounding and may replace either term; integers are off by half a step."""
    api = require_gpu()
    x, r, w = rows_of(normal((rows, dim), kind, 3)), rows_of(normal((rows, dim), kind, 4, 2.0), 1), normal((dim,), kind, 5)
    h, y = reference(x, r, w, float(np.float32(1e-5)))
    total = {"x": x, "residual": r, "new": rows_of(torch.zeros_like(x), 2), None: None}[where]
    out = rows_of(torch.zeros(rows, dim, dtype=torch.int8, device="cuda"), 1)
    scales = torch.zeros(rows, device="cuda")
    api.mxnorm_run(fmt_of(api, kind), x, out, scales, api.MX_INT8, weight=w, eps=1e-5, residual=r, total=total)
    if total is not None:
        assert torch.equal(total, h)
    most = np.abs(y).max(-1)
    rel = relative(dim)
    assert np.all(np.abs(f64(scales) - most / 127) <= most / 127 * (rel + 3 * U32))
    q = f64(out)
    err = np.abs(q - 127 * y / most[:, None])
    say(f"int8 {kind} {rows}x{dim}: worst {err.max():.5f} steps")
    assert err.max() <= 0.5 + 127 * (rel + 4 * U32) and np.abs(q).max() <= 127
    assert np.all(np.abs(q).max(-1) == 127)
    assert bool((torch.as_strided(out, (rows, out.stride(0) - dim), (out.stride(0), 1), dim) == 0x5A).all())


@pytest.mark.parametrize("fmt,bits,top,most,least", [("MX_E4M3", 3, 8, 448.0, -9), ("MX_E5M2", 2, 15, 57344.0, -16)])
@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,dim", [(1, 32), (1030, 96), (5, 4096), (1030, 4096), (2, 8192), (1030, 8192), (2, 40000)])
def test_norm_blocks(fmt, bits, top, most, least, kind, rows, dim):
    api = require_gpu()
    x, r, w = normal((rows, dim), kind, 6), normal((rows, dim), kind, 7, 30.0), normal((dim,), kind, 8)
    codes, scales = torch.full((rows, dim), 0x5A, dtype=torch.uint8, device="cuda"), torch.full((rows, dim // 32), 0x5A, dtype=torch.uint8, device="cuda")
    api.mxnorm_run(fmt_of(api, kind), x, codes, scales, getattr(api, fmt), weight=w, eps=1e-5, residual=r)
    _, y = reference(x, r, w, float(np.float32(1e-5)))
    rel = relative(dim)
    b, e = np.abs(y).reshape(rows, -1, 32).max(-1), host(scales).astype(int) - 127
    lo, hi = (np.floor(np.log2(b * (1 + s * rel))) - top for s in (-1, 1))
    assert np.all((e == lo) | (e == hi))
    step = np.repeat(2.0 ** e, 32, axis=1)
    kind8 = torch.float8_e4m3fn if fmt == "MX_E4M3" else torch.float8_e5m2
    got = f64(codes.view(kind8)) * step
    want = np.clip(y, -most * step, most * step)
    bound = np.maximum(np.abs(y) * 2.0 ** -(bits + 1), 2.0 ** (least - 1) * step) * (1 + 4 * rel) + np.abs(y) * rel
    err = (np.abs(got - want) / bound).max()
    say(f"{fmt} {kind} {rows}x{dim}: worst error / bound {err:.3f}")
    assert err <= 1.0


@pytest.mark.parametrize("fmt,top", [("MX_E4M3", 8), ("MX_E5M2", 15)])
@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,dim", [(1, 64), (1030, 96), (3, 4096), (1100, 2048), (2, 8192), (2, 40000)])
def test_scales_at_powers_of_two(fmt, top, kind, rows, dim):
    """A block's scale is that of y before its rounding: elements +-c of one size have y = c / sqrt(c^2 + eps), which is below 1 by less than fp32 holds with a small
    eps, and 1 without one."""
    api = require_gpu()
    x = torch.where(torch.arange(rows * dim, device="cuda").reshape(rows, dim) % 3 == 0, -2.0, 2.0).to({"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[kind])
    codes, scales = torch.zeros(rows, dim, dtype=torch.uint8, device="cuda"), torch.zeros(rows, dim // 32, dtype=torch.uint8, device="cuda")
    for eps, e in ((1e-9, -1), (0.0, 0)):
        api.mxnorm_run(fmt_of(api, kind), x, codes, scales, getattr(api, fmt), eps=eps)
        assert bool((scales == 127 + e - top).all())
        y = codes.view(torch.float8_e4m3fn if fmt == "MX_E4M3" else torch.float8_e5m2).float() * 2.0 ** (e - top)
        # scaled to 2^(top + 1) less a little, which is cut to the largest element, 1.75 * 2^top
        assert torch.equal(y, x.float() * (0.5 if e == 0 else 0.4375))


def awkward(dim):
    """Rows of zeros, subnormals, one element, the largest values, infinities and NaN."""
    g = np.random.Generator(np.random.PCG64(9))
    x = g.standard_normal((16, dim)).astype(np.float32)
    x[0] = 0
    x[1] *= np.float32(1e-40)
    x[2, 1:] = 0
    x[3] *= np.float32(1e38)
    x[4, dim // 2] = np.inf
    x[5, dim - 1] = np.nan
    x[6] *= 2.0 ** g.integers(-40, 40, dim).astype(np.float32)
    x[7] = np.float32(3.4028235e38)
    x[8] = np.float32(1e-45)
    x[9] *= np.float32(1e-30)
    x[10] = np.where(g.random(dim) < 0.5, 448.0, -464.0)
    x[11] = -0.0
    x[12] *= np.float32(1e20)
    x[13, 0] = -np.inf
    x[14] = np.exp2(g.integers(-140, 120, dim)).astype(np.float32)
    x[15] = np.round(x[15] * 4) / 4
    return x


@pytest.mark.parametrize("fmt", ["MX_E4M3", "MX_E5M2"])
@pytest.mark.parametrize("dim", [32, 4128, 40000])
def test_quant_rows_is_pack(fmt, dim):
    """Codes and scales are mx_pack_run's, bit for bit, of every row."""
    api = require_gpu()
    x = np.concatenate([awkward(dim)] + [awkward(dim)[6:7] * np.float32(2.0) ** k for k in range(-60, 60, 7)])
    want = [torch.zeros(x.shape, dtype=torch.uint8, device="cuda"), torch.zeros((len(x), dim // 32), dtype=torch.uint8, device="cuda")]
    got = [torch.full_like(t, 0x5A) for t in want]
    api.mx_pack_run(getattr(api, fmt), dev(x), len(x), dim, *want)
    api.mxquant_rows_run(api.MX_F32, dev(x), *got, getattr(api, fmt))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dim", [31, 4096])
def test_quant_rows_int8(kind, dim):
    api = require_gpu()
    x = rows_of(torch.from_numpy(awkward(dim)).to(TORCH[kind]).cuda())
    z = f64(x)
    out, scales = rows_of(torch.zeros(x.shape, dtype=torch.int8, device="cuda")), torch.full((16,), 7.0, device="cuda")
    api.mxquant_rows_run(fmt_of(api, kind), x, out, scales, api.MX_INT8)
    q, s = f64(out), f64(scales)
    for i in range(16):
        if not np.isfinite(z[i]).all():
            assert np.isnan(s[i]) and not q[i].any(), i
            continue
        most = np.abs(z[i]).max()
        assert abs(s[i] - most / 127) <= most / 127 * 2 * U32 + TINY["f32"], i
        if most == 0:
            assert s[i] == 0 and not q[i].any(), i
        else:
            assert np.abs(q[i] - 127 * z[i] / most).max() <= 0.5 + 127 * 4 * U32, i


@pytest.mark.parametrize("dim", [24, 4096, 40000])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-20, 1e-6])
def test_norm_of_far_values(dim, eps):
    """fp32 rows whose squares overflow or vanish have their norm all the same; infinities and NaN act as in the formula."""
    api = require_gpu()
    x = awkward(dim)
    eps32 = float(np.float32(eps))
    out = torch.zeros(x.shape, device="cuda")
    api.mxnorm_run(api.MX_F32, dev(x), out, None, api.MX_F32, eps=eps)
    got, z = f64(out), x.astype(np.float64)
    q, s = torch.zeros(x.shape, dtype=torch.int8, device="cuda"), torch.zeros(16, device="cuda")
    q = rows_of(q)
    api.mxnorm_run(api.MX_F32, dev(x), q, s, api.MX_INT8, eps=eps)
    s, q = f64(s), f64(q)
    for i in range(16):
        if np.isnan(z[i]).any():
            assert np.isnan(got[i]).all() and np.isnan(s[i]) and not q[i].any(), i
            continue
        if np.isinf(z[i]).any():
            assert np.all(np.isnan(got[i]) == np.isinf(z[i])) and not got[i][np.isfinite(z[i])].any() and np.isnan(s[i]), i
            continue
        mean = (z[i] * z[i]).mean() + eps32
        if mean == 0:
            assert np.isnan(got[i]).all() and np.isnan(s[i]), i
            continue
        y = z[i] / np.sqrt(mean)
        # scaling by a power of two may cost elements 2^-126 below the largest one their last bits
        bound = np.abs(y) * (relative(dim) + U32) + 2.0 ** -126 + 2.0 ** -126 * np.abs(y).max()
        assert np.all(np.abs(got[i] - y) <= bound), (i, (np.abs(got[i] - y) / bound).max())
        most = np.abs(y).max()
        assert abs(s[i] - most / 127) <= most / 127 * (relative(dim) + 4 * U32) + 2.0 ** -126, i
        if most > 2.0 ** -100:
            assert np.abs(q[i] - 127 * y / most).max() <= 0.5 + 127 * (relative(dim) + 4 * U32) + 1e-4, i


def test_norm_streams_and_graph():
    """On another stream, and captured into a graph that is replayed with new inputs."""
    api = require_gpu()
    x, w = normal((37, 512), "f16", 11), normal((512,), "f16", 12)
    want, got = torch.zeros_like(x), torch.zeros_like(x)
    api.mxnorm_run(api.MX_F16, x, want, None, api.MX_F16, weight=w)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    api.mxnorm_run(api.MX_F16, x, got, None, api.MX_F16, weight=w, stream=stream)
    stream.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.mxnorm_run(api.MX_F16, x, got, None, api.MX_F16, weight=w)
    for seed in (13, 14, 15):
        x.copy_(normal((37, 512), "f16", seed))
        graph.replay()
        api.mxnorm_run(api.MX_F16, x, want, None, api.MX_F16, weight=w)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
