"""The product of 8-bit integers with scales per row of each operand, against exact sums."""
import numpy as np
import pytest
import torch

from cache_common import TORCH, f64, fmt_of
from cache_reference import HALF_STEP, TINY, U32
from gpu_common import dev, require_gpu, say

pytestmark = pytest.mark.gpu
COUNTERS = 16384


def codes(rows, K, seed, pad=0, lo=-128):
    """Random bytes in rows of whole 16-byte pieces and `pad` more; what is between the rows is not zero."""
    g = torch.Generator().manual_seed(seed)
    wide = -(-K // 16) * 16 + 16 * pad
    return torch.randint(lo, 128, (rows, wide), generator=g, dtype=torch.int8).cuda()[:, :K]


def scales(n, seed):
    return torch.rand(n, generator=torch.Generator().manual_seed(seed)).cuda() * 0.1 + 0.001


def workspace(M, N, K):
    return torch.zeros(max(16, require_gpu().mxgemm_i8_workspace_size(M, N, K)), dtype=torch.uint8, device="cuda")


def want_of(A, SA, B, SB, bias=None, relu=False):
    c = (A.double() @ B.double().t().contiguous()) * SA.double()[:, None] * SB.double()
    if bias is not None:
        c = c + bias.double()
    return f64(torch.clamp(c, min=0) if relu else c)


def check(kind, C, want, bias=None):
    """Three roundings to fp32 (the sum, the scales' product, theirs), one of the bias' sum, and the result's."""
    size = np.abs(want) if bias is None else np.abs(want) + 2 * np.abs(f64(bias))
    err = np.abs(f64(C) - want) / (np.abs(want) * HALF_STEP[kind] * 1.01 + 4 * U32 * size + TINY[kind])
    assert np.all(np.isfinite(f64(C))) and err.max() <= 1.0, err.max()
    return err.max()


def run(M, N, K, kind="f16", seed=0, pad=(0, 0), c_stride=None, bias=False, relu=False, ws=True):
    api = require_gpu()
    A, B, SA, SB = codes(M, K, seed, pad[0]), codes(N, K, seed + 1, pad[1]), scales(M, seed + 2), scales(N, seed + 3)
    b = (torch.randn(N, generator=torch.Generator().manual_seed(seed + 4)) * 20).to(TORCH[kind]).cuda() if bias else None
    C = torch.full((M, c_stride or N), float("nan"), dtype=TORCH[kind], device="cuda")
    w = workspace(M, N, K) if ws else None
    say(f"i8 {M}x{N}x{K} {kind} workspace {0 if w is None else w.numel()}")
    api.mxgemm_i8_run(A, SA, B, SB, C[:, :N], fmt_of(api, kind), bias=b, flags=api.MXGEMM_RELU if relu else 0, workspace=w)
    worst = check(kind, C[:, :N], want_of(A, SA, B, SB, b, relu), b)
    assert C[:, N:].isnan().all()
    if w is not None and w.numel() > 16:
        assert not bool(w[:COUNTERS].any()), "counters not back at zero"
    say(f"worst error / bound {worst:.3f}")
    return C


@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 64])
@pytest.mark.parametrize("N,K", [(1, 1), (3, 15), (16, 16), (33, 17), (100, 64), (130, 65), (48, 1000), (1000, 4099), (4112, 515), (16400, 272)])
def test_few_rows(M, N, K):
    run(M, N, K, "f16", M + N + K, pad=(M % 3, N % 2))


@pytest.mark.parametrize("M", [65, 128, 131, 300])
@pytest.mark.parametrize("N,K", [(1, 1), (5, 31), (128, 128), (129, 127), (257, 130), (1003, 2741), (640, 1024)])
def test_tiles(M, N, K):
    run(M, N, K, "bf16", M + N + K, pad=(N % 2, M % 3))


@pytest.mark.parametrize("M,N,K", [(2048, 6400, 40), (3500, 3700, 300), (4096, 3328, 129), (70000, 257, 16), (257, 70000, 100)])
def test_large_tiles(M, N, K):
    run(M, N, K, "f16", 1)


@pytest.mark.parametrize("K", [1, 16, 128, 129, 257, 400, 513, 1157])
@pytest.mark.parametrize("M,N,kind", [(1500, 2100, "f16"), (1000, 3201, "f32"), (2200, 3001, "bf16"), (1800, 3500, "f32"), (3500, 3701, "f16"), (3300, 3800, "f32")])
def test_rings(M, N, kind, K):
    """One to ten slots of K through the rings of tiles 128 wide, for as many workgroups as there are CUs and for more, and 256 wide."""
    run(M, N, K, kind, K, pad=(K % 2, K % 3), bias=bool(K % 2), relu=bool(K % 3))


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(3, 70, 200), (100, 200, 1500), (2100, 6200, 160)])
def test_types_bias_relu(kind, M, N, K):
    for bias, relu in ((True, False), (False, True), (True, True)):
        run(M, N, K, kind, 5, bias=bias, relu=relu)


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K,stride", [(5, 64, 64, 72), (5, 64, 64, 65), (5, 61, 64, 77), (150, 192, 96, 200), (150, 192, 96, 195), (150, 131, 96, 131), (2048, 6401, 64, 6403)])
def test_strides_of_c(kind, M, N, K, stride):
    run(M, N, K, kind, 7, c_stride=stride)


@pytest.mark.parametrize("M,N,K", [(1, 512, 8192), (16, 48, 16000), (40, 260, 5000), (64, 1024, 4096), (70, 128, 3000), (200, 384, 9001), (300, 1000, 1024)])
def test_split_is_the_same(M, N, K):
    """Workgroups that share K give the bits of those that do not; one workspace serves them all, call after call."""
    api = require_gpu()
    need = api.mxgemm_i8_workspace_size(M, N, K)
    assert need > COUNTERS
    A, B, SA, SB = codes(M, K, 1), codes(N, K, 2), scales(M, 3), scales(N, 4)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    whole, split = (torch.full((M, N), float("nan"), device="cuda") for _ in range(2))
    api.mxgemm_i8_run(A, SA, B, SB, whole, api.MX_F32)
    check("f32", whole, want_of(A, SA, B, SB))
    for i in range(3):
        split.fill_(float("nan"))
        api.mxgemm_i8_run(A, SA, B, SB, split, api.MX_F32, workspace=ws)
        other = torch.zeros(9, 50, device="cuda")
        api.mxgemm_i8_run(codes(9, 3000, 5), scales(9, 6), codes(50, 3000, 7), scales(50, 8), other, api.MX_F32, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(whole, split) and not bool(ws[:COUNTERS].any())
    split.fill_(float("nan"))
    api.mxgemm_i8_run(A, SA, B, SB, split, api.MX_F32, workspace=ws, workspace_bytes=need - 1)  # too small: not used
    torch.cuda.synchronize()
    assert torch.equal(whole, split)


@pytest.mark.parametrize("M", [1, 130])
def test_largest_sums(M):
    """K of the bound, all products 2^14: the sum is 2^31 - 2^14."""
    api = require_gpu()
    K, N = api.MXGEMM_I8_MAX_K, 20
    A, B = (torch.full((r, 131072), -128, dtype=torch.int8, device="cuda")[:, :K] for r in (M, N))
    ones = torch.ones(max(M, N), device="cuda")
    C = torch.zeros(M, N, device="cuda")
    for ws in (None, workspace(M, N, K)):
        api.mxgemm_i8_run(A, ones[:M], B, ones[:N], C, api.MX_F32, workspace=ws)
        assert bool((C.double() == float(np.float32(K * 16384))).all())


def test_scales_of_nothing_and_nan():
    """Zero scales give zeros, NaN scales rows and columns of NaN (0 under ReLU), infinities signed ones."""
    api = require_gpu()
    A, B, SA, SB = codes(70, 100, 1), codes(40, 100, 2), scales(70, 3), scales(40, 4)
    SA[3], SA[69], SB[7] = 0.0, float("nan"), float("inf")
    for relu in (False, True):
        C = torch.zeros(70, 40, device="cuda")
        api.mxgemm_i8_run(A, SA, B, SB, C, api.MX_F32, flags=api.MXGEMM_RELU if relu else 0)
        c = f64(C)
        s = f64(A.double() @ B.double().t().contiguous())
        assert np.all(c[3, np.arange(40) != 7] == 0)
        assert np.all(c[69] == 0) if relu else np.isnan(c[69]).all()
        col = np.array([i for i in range(70) if i not in (3, 69)])
        assert np.all(c[col, 7] == np.where(s[col, 7] > 0, np.inf, 0.0 if relu else -np.inf))


def test_streams_and_graph():
    api = require_gpu()
    M, N, K = 40, 260, 5000
    A, B, SA, SB = codes(M, K, 1), codes(N, K, 2), scales(M, 3), scales(N, 4)
    C, ws = torch.zeros(M, N, dtype=torch.float16, device="cuda"), workspace(M, N, K)
    want = torch.zeros_like(C)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.mxgemm_i8_run(A, SA, B, SB, C, api.MX_F16, workspace=ws)
    for seed in (5, 6, 7):
        A.copy_(codes(M, K, seed))
        C.fill_(float("nan"))
        graph.replay()
        api.mxgemm_i8_run(A, SA, B, SB, want, api.MX_F16)
        torch.cuda.synchronize()
        assert torch.equal(C, want)
    stream = torch.cuda.Stream()
    C.fill_(float("nan"))
    torch.cuda.synchronize()
    api.mxgemm_i8_run(A, SA, B, SB, C, api.MX_F16, workspace=ws, stream=stream)
    stream.synchronize()
    assert torch.equal(C, want)


@pytest.mark.parametrize("M", [5, 200])
def test_normalised_rows_times_quantised_weights(M):
    """The chain of a layer: norm with the residual to int8, weights quantised by channel, their product. An element of y is off by half its
    row's step, one of w by half its channel's; a product's errors are independent, and six times their standard deviation bounds all of them."""
    api = require_gpu()
    N, K = 300, 1024
    g = torch.Generator().manual_seed(3)
    x, r, w = (torch.randn(s, generator=g).half().cuda() for s in ((M, K), (M, K), (N, K)))
    total = torch.zeros_like(x)
    a, sa = torch.zeros((M, K), dtype=torch.int8, device="cuda"), torch.zeros(M, device="cuda")
    b, sb = torch.zeros((N, K), dtype=torch.int8, device="cuda"), torch.zeros(N, device="cuda")
    C = torch.zeros(M, N, dtype=torch.float16, device="cuda")
    api.mxquant_rows_run(api.MX_F16, w, b, sb, api.MX_INT8)
    api.mxnorm_run(api.MX_F16, x, a, sa, api.MX_INT8, eps=1e-5, residual=r, total=total)
    api.mxgemm_i8_run(a, sa, b, sb, C, api.MX_F16, workspace=workspace(M, N, K))
    h = total.double()
    y = h / (h.pow(2).mean(-1, keepdim=True) + 1e-5).sqrt()
    want = f64(y @ w.double().t().contiguous())
    y, w = f64(y), f64(w)
    step_a, step_b = np.abs(y).max(1) / 127, np.abs(w).max(1) / 127
    sigma = np.sqrt((step_a ** 2 / 12)[:, None] * (w ** 2).sum(1) + (step_b ** 2 / 12) * (y ** 2).sum(1)[:, None] + K * np.outer(step_a, step_b) ** 2 / 144)
    err = np.abs(f64(C) - want) / (6 * sigma + 2.0 ** -11 * np.abs(want))
    say(f"chain of {M} rows: worst error / bound {err.max():.3f}")
    assert err.max() <= 1.0


@pytest.mark.parametrize("few", [1, 16, 17, 64, 65, 128, 129])
@pytest.mark.parametrize("many,K", [(24449, 100), (48897, 65), (70001, 160), (128256, 32)])
def test_few_rows_of_many_columns(few, many, K):
    """A vocabulary's projection of a few tokens, and as many rows by few columns."""
    run(few, many, K, "f16", few + many + K, pad=(few % 3, many % 2))
    run(many, few, K, "bf16", few + many + K, bias=True, relu=True)
