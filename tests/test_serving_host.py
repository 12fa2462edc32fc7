"""Argument checks of the norm, the 8-bit product and the step planner: statuses of the C entry points and of the binding, without a GPU. Nothing
is queued where a call is refused."""
import ctypes

import pytest
import torch

api = pytest.importorskip("block_scaled_quantized_amd.api")
lib = api._lib
P = 0x10000  # an address that is never read: calls are refused, or end at the check of the device


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64)]


class StepArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("seqs", "cols", "page_size", "pages", "max_tokens")] + \
        [(n, ctypes.c_void_p) for n in ("table", "lengths", "wants", "kept", "free_pages", "n_free", "lengths_out", "n_free_out", "offsets", "seq",
                                        "positions", "slots", "status")]


def rows(data=P, stride=64):
    return ctypes.byref(Rows(data, stride))


def norm(f=api.MX_F16, n=4, dim=64, x=rows(), residual=None, total=None, weight=P, eps=1e-6, fmt=api.MX_INT8, out=rows(), scales=P):
    return lib.mxnorm_run(f, n, dim, x, residual, total, weight, eps, fmt, out, scales, None)


@pytest.mark.parametrize("status,args", [
    (api.MX_ERR_FORMAT, dict(f=api.MX_E4M3)), (api.MX_ERR_FORMAT, dict(fmt=api.MX_E2M1)), (api.MX_ERR_FORMAT, dict(fmt=api.MX_BF16)),
    (api.MX_ERR_SHAPE, dict(n=-1)), (api.MX_ERR_SHAPE, dict(dim=0)), (api.MX_ERR_SHAPE, dict(dim=(1 << 20) + 1)), (api.MX_ERR_SHAPE, dict(n=(1 << 20) + 1)),
    (api.MX_ERR_SHAPE, dict(dim=48, fmt=api.MX_E4M3)), (api.MX_ERR_SHAPE, dict(dim=40, fmt=api.MX_E5M2)),
    (api.MX_ERR_SHAPE, dict(eps=-1.0)), (api.MX_ERR_SHAPE, dict(eps=float("nan"))), (api.MX_ERR_SHAPE, dict(eps=float("inf"))),
    (api.MX_ERR_NULL, dict(x=None)), (api.MX_ERR_NULL, dict(out=None)), (api.MX_ERR_NULL, dict(scales=None)), (api.MX_ERR_NULL, dict(x=rows(None))),
    (api.MX_ERR_NULL, dict(out=rows(None))), (api.MX_ERR_NULL, dict(total=rows())), (api.MX_ERR_NULL, dict(residual=rows(None))),
    (api.MX_ERR_SHAPE, dict(x=rows(P, 56))), (api.MX_ERR_SHAPE, dict(x=rows(P, 68))), (api.MX_ERR_SHAPE, dict(out=rows(P, 72))),
    (api.MX_ERR_SHAPE, dict(residual=rows(P, 65))), (api.MX_ERR_SHAPE, dict(residual=rows(), total=rows(P, 66))),
    (api.MX_ERR_ALIGN, dict(x=rows(P + 8))), (api.MX_ERR_ALIGN, dict(out=rows(P + 8))), (api.MX_ERR_ALIGN, dict(weight=P + 2)), (api.MX_ERR_ALIGN, dict(scales=P + 4)),
    (api.MX_OK, dict(n=0)), (api.MX_OK, dict(n=0, x=rows(None), scales=None)),
])
def test_norm_refusals(status, args):
    assert norm(**args) == status


def test_quant_refusals():
    run = lambda f=api.MX_F16, n=4, dim=64, x=rows(), fmt=api.MX_INT8, out=rows(), scales=P: lib.mxquant_rows_run(f, n, dim, x, fmt, out, scales, None)  # noqa: E731
    assert run(fmt=api.MX_F16) == api.MX_ERR_FORMAT and run(f=api.MX_INT8) == api.MX_ERR_FORMAT
    assert run(dim=33, fmt=api.MX_E4M3) == api.MX_ERR_SHAPE and run(scales=None) == api.MX_ERR_NULL
    assert run(out=rows(P + 1)) == api.MX_ERR_ALIGN and run(n=0) == api.MX_OK


def gemm(M=4, N=8, K=64, A=rows(), SA=P, B=rows(), SB=P, bias=None, fc=api.MX_F16, C=rows(), flags=0, ws=None, size=0):
    return lib.mxgemm_i8_run(M, N, K, A, SA, B, SB, bias, fc, C, flags, ws, size, None)


@pytest.mark.parametrize("status,args", [
    (api.MX_ERR_FORMAT, dict(fc=api.MX_INT8)), (api.MX_ERR_FORMAT, dict(flags=2)), (api.MX_ERR_SHAPE, dict(M=-1)), (api.MX_ERR_SHAPE, dict(N=0)),
    (api.MX_ERR_SHAPE, dict(K=0)), (api.MX_ERR_SHAPE, dict(K=131072, A=rows(P, 131072), B=rows(P, 131072))), (api.MX_ERR_SHAPE, dict(M=(1 << 20) + 1)),
    (api.MX_ERR_SHAPE, dict(N=(1 << 20) + 1, C=rows(P, 1 << 21))), (api.MX_ERR_SHAPE, dict(A=rows(P, 48))), (api.MX_ERR_SHAPE, dict(A=rows(P, 72))),
    (api.MX_ERR_SHAPE, dict(B=rows(P, 65))), (api.MX_ERR_SHAPE, dict(B=rows(P, 1 << 21))), (api.MX_ERR_SHAPE, dict(C=rows(P, 7))),
    (api.MX_ERR_NULL, dict(A=None)), (api.MX_ERR_NULL, dict(A=rows(None))), (api.MX_ERR_NULL, dict(SA=None)), (api.MX_ERR_NULL, dict(B=rows(None))),
    (api.MX_ERR_NULL, dict(SB=None)), (api.MX_ERR_NULL, dict(C=None)), (api.MX_ERR_NULL, dict(C=rows(None))),
    (api.MX_ERR_ALIGN, dict(A=rows(P + 8))), (api.MX_ERR_ALIGN, dict(SA=P + 4)), (api.MX_ERR_ALIGN, dict(B=rows(P + 1))), (api.MX_ERR_ALIGN, dict(SB=P + 8)),
    (api.MX_ERR_ALIGN, dict(C=rows(P + 2))), (api.MX_ERR_ALIGN, dict(bias=P + 2)), (api.MX_ERR_ALIGN, dict(ws=P + 4, size=1 << 20)), (api.MX_OK, dict(M=0)),
])
def test_gemm_refusals(status, args):
    assert gemm(**args) == status


def test_gemm_workspace_sizes():
    size = api.mxgemm_i8_workspace_size
    assert size(0, 8, 64) == size(4, 0, 64) == size(4, 8, 131072) == 0
    assert size(1, 64, 8192) > 16384 and size(8192, 8192, 512) == 0
    with pytest.raises(api.MXError):
        size(1 << 32, 8, 64)


def step(**args):
    a = dict(seqs=2, cols=4, page_size=16, pages=10, max_tokens=8, slots=None, kept=None)
    a.update({n: P for n, _ in StepArgs._fields_[5:] if n not in a})
    a.update(args)
    return lib.mxkv_step_run(ctypes.byref(StepArgs(**a)), None)


@pytest.mark.parametrize("status,args", [
    (api.MX_ERR_SHAPE, dict(seqs=-1)), (api.MX_ERR_SHAPE, dict(seqs=(1 << 20) + 1)), (api.MX_ERR_SHAPE, dict(cols=0)), (api.MX_ERR_SHAPE, dict(page_size=0)),
    (api.MX_ERR_SHAPE, dict(pages=0)), (api.MX_ERR_SHAPE, dict(max_tokens=-1)), (api.MX_ERR_SHAPE, dict(max_tokens=(1 << 20) + 1)),
    (api.MX_ERR_SHAPE, dict(cols=1 << 27)), (api.MX_ERR_SHAPE, dict(pages=1 << 20, page_size=2048)), (api.MX_OK, dict(seqs=0, table=None)),
] + [(api.MX_ERR_NULL, {n: None}) for n in ("table", "lengths", "wants", "free_pages", "n_free", "lengths_out", "n_free_out", "offsets", "seq", "positions", "status")])
def test_step_refusals(status, args):
    assert step(**args) == status
    assert lib.mxkv_step_run(None, None) == api.MX_ERR_NULL


def refused(status, call, *args, **kw):
    with pytest.raises(api.MXError) as e:
        call(*args, **kw)
    assert e.value.status == status


def t(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refusals_of_the_norm():
    x, out, s = t(4, 64), t(4, 64, dtype=torch.int8), t(4, dtype=torch.float32)
    run = lambda **kw: api.mxnorm_run(**{**dict(f=api.MX_F16, x=x, out=out, scales=s, fmt=api.MX_INT8), **kw})  # noqa: E731
    refused(api.MX_ERR_FORMAT, run, f=api.MX_BF16)
    refused(api.MX_ERR_FORMAT, run, fmt=api.MX_F16)
    refused(api.MX_ERR_FORMAT, run, out=t(4, 64, dtype=torch.float8_e4m3fn))
    refused(api.MX_ERR_FORMAT, run, scales=t(4))
    refused(api.MX_ERR_FORMAT, run, weight=t(64, dtype=torch.float32))
    refused(api.MX_ERR_FORMAT, run, f=1 << 40)
    refused(api.MX_ERR_SHAPE, run, x=t(4, 32))
    refused(api.MX_ERR_SHAPE, run, x=t(64, 4).t())
    refused(api.MX_ERR_SHAPE, run, scales=t(5, dtype=torch.float32))
    refused(api.MX_ERR_SHAPE, run, weight=t(63))
    refused(api.MX_ERR_SHAPE, run, weight=t(128)[::2])
    refused(api.MX_ERR_SHAPE, run, residual=t(3, 64))
    refused(api.MX_ERR_SHAPE, run, fmt=api.MX_E4M3, out=t(4, 64, dtype=torch.uint8), scales=t(4, 1, dtype=torch.uint8))
    with pytest.raises(TypeError):
        run()  # tensors in host memory
    with pytest.raises(TypeError):
        run(x=None)
    quant = lambda **kw: api.mxquant_rows_run(**{**dict(f=api.MX_F16, x=x, out=out, scales=s, fmt=api.MX_INT8), **kw})  # noqa: E731
    refused(api.MX_ERR_FORMAT, quant, out=x)
    refused(api.MX_ERR_SHAPE, quant, out=t(4, 60, dtype=torch.int8))
    with pytest.raises(TypeError):
        quant()


def test_binding_refusals_of_the_product():
    A, B, C, sa, sb = t(4, 64, dtype=torch.int8), t(8, 64, dtype=torch.int8), t(4, 8), t(4, dtype=torch.float32), t(8, dtype=torch.float32)
    run = lambda **kw: api.mxgemm_i8_run(**{**dict(A=A, SA=sa, B=B, SB=sb, C=C, fc=api.MX_F16), **kw})  # noqa: E731
    refused(api.MX_ERR_FORMAT, run, A=t(4, 64, dtype=torch.uint8))
    refused(api.MX_ERR_FORMAT, run, C=t(4, 8, dtype=torch.bfloat16))
    refused(api.MX_ERR_FORMAT, run, fc=api.MX_INT8)
    refused(api.MX_ERR_FORMAT, run, bias=t(8, dtype=torch.float32))
    refused(api.MX_ERR_FORMAT, run, flags=-1)
    refused(api.MX_ERR_SHAPE, run, B=t(8, 32, dtype=torch.int8))
    refused(api.MX_ERR_SHAPE, run, C=t(4, 9))
    refused(api.MX_ERR_SHAPE, run, SA=t(3, dtype=torch.float32))
    refused(api.MX_ERR_SHAPE, run, SB=t(8))
    refused(api.MX_ERR_SHAPE, run, bias=t(7))
    refused(api.MX_ERR_SHAPE, run, workspace=t(64, dtype=torch.uint8), workspace_bytes=65)
    # a last row whose memory ends before its last 16-byte piece does
    refused(api.MX_ERR_SHAPE, run, A=torch.as_strided(t(3 * 64 + 50, dtype=torch.int8), (4, 50), (64, 1)), B=t(8, 64, dtype=torch.int8)[:, :50])
    with pytest.raises(TypeError):
        run()


def test_binding_refusals_of_the_step():
    i = lambda *shape: torch.zeros(shape, dtype=torch.int32)  # noqa: E731
    base = dict(page_size=16, table=i(2, 4), lengths=i(2), wants=i(2), free=i(10), n_free=i(1), offsets=i(3), seq=i(8), positions=i(8), slots=i(8), status=i(1))
    run = lambda **kw: api.mxkv_step_run(**{**base, **kw})  # noqa: E731
    for name, bad in dict(table=i(8), lengths=i(3), wants=i(2).long(), free=i(2, 5), n_free=i(2), offsets=i(2), positions=i(7), slots=i(9), kept=i(1),
                          lengths_out=i(3), n_free_out=i(2)).items():
        refused(api.MX_ERR_SHAPE, lambda: run(**{name: bad}))
    refused(api.MX_ERR_SHAPE, lambda: run(status=i(0)))
    refused(api.MX_ERR_SHAPE, run, page_size=1 << 33)
    with pytest.raises(TypeError):
        run()


def cache_of(fmt=api.MX_F16, pages=8, page=16, heads=2, dim=64):
    k = torch.zeros(pages, heads, page, dim, dtype=torch.float16)
    return api.KVCache(fmt, k, k)


class Groups(ctypes.Structure):
    _fields_ = [("first", ctypes.c_void_p), ("shared", ctypes.c_void_p), ("count", ctypes.c_int), ("max_shared", ctypes.c_int)]


def prefix(groups=(P, P, 2, 100), f=api.MX_F16, heads=4, max_len=128, window=0, softcap=0.0, scale=1.0, seqs=3, lengths=P, ws=None, table=P, dim=64):
    c = cache_of(dim=dim)
    q = api._Heads(P, heads, heads * dim, dim)
    t, o = api._Table(table, seqs, 8), api._AttnOpts(scale, softcap, window)
    g = None if groups is None else ctypes.byref(Groups(*groups))
    return lib.mxattn_prefix_run(ctypes.byref(c.c), f, ctypes.byref(q), ctypes.byref(q), None, ctypes.byref(t), lengths, g, max_len, ctypes.byref(o), ws, 0, None)


@pytest.mark.parametrize("status,args", [
    (api.MX_ERR_NULL, dict(groups=None)), (api.MX_ERR_NULL, dict(groups=(None, P, 2, 100))), (api.MX_ERR_NULL, dict(groups=(P, None, 2, 100))),
    (api.MX_ERR_SHAPE, dict(groups=(P, P, -1, 100))), (api.MX_ERR_SHAPE, dict(groups=(P, P, 1025, 100))), (api.MX_ERR_SHAPE, dict(groups=(P, P, 2, -1))),
    (api.MX_ERR_SHAPE, dict(window=16)), (api.MX_ERR_SHAPE, dict(max_len=0)), (api.MX_ERR_SHAPE, dict(heads=3)), (api.MX_ERR_SHAPE, dict(softcap=-1.0)),
    (api.MX_ERR_SHAPE, dict(scale=float("nan"))), (api.MX_ERR_FORMAT, dict(f=api.MX_BF16)), (api.MX_ERR_FORMAT, dict(f=api.MX_F32)), (api.MX_ERR_NULL, dict(lengths=None)),
    (api.MX_ERR_NULL, dict(table=None)), (api.MX_ERR_ALIGN, dict(ws=P + 8)), (api.MX_OK, dict(seqs=0, table=None)),
])
def test_prefix_refusals(status, args):
    assert prefix(**args) == status


def test_prefix_workspace_sizes():
    size, c = api.mxattn_prefix_workspace_size, cache_of()
    assert size(c, 0, 4, 2, 100, 100) == size(c, 3, 3, 2, 100, 100) == size(c, 3, 4, -1, 100, 100) == size(c, 3, 4, 1025, 100, 100) == size(c, 3, 4, 2, 100, -1) == 0
    # nothing to share, or too little
    for args in ((1, 4, 1, 50000, 50000), (9, 4, 0, 50000, 50000), (9, 4, 9, 50000, 50000), (9, 4, 2, 50000, 63), (9, 4, 2, 63, 50000), (9, 4, 2, 50000, 2000)):
        assert size(c, *args) == api.mxattn_decode_workspace_size(c, *args[:2], args[3])
    assert size(c, 9, 4, 2, 50000, 40000) > api.mxattn_decode_workspace_size(c, 9, 4, 50000)
    with pytest.raises(api.MXError):
        size(c, 9, 4, 2, 1 << 40, 64)


def test_binding_refusals_of_the_prefix():
    i = lambda *shape: torch.zeros(shape, dtype=torch.int32)  # noqa: E731
    base = dict(cache=cache_of(), f=api.MX_F16, q=t(3, 4, 64), out=t(3, 4, 64), table=i(3, 8), lengths=i(3), max_len=100, first=i(3), shared=i(2), max_shared=50, scale=1.0)
    run = lambda **kw: api.mxattn_prefix_run(**{**base, **kw})  # noqa: E731
    for bad in (dict(out=t(3, 5, 64)), dict(q=t(3, 4, 32), out=t(3, 4, 32)), dict(table=i(2, 8)), dict(lengths=i(4)), dict(first=i(2)), dict(first=i(3).long()),
                dict(shared=i(2, 1)), dict(max_shared=1 << 31), dict(max_len=1 << 40), dict(lse=t(3, 4)), dict(workspace=t(8, dtype=torch.uint8), workspace_bytes=9)):
        refused(api.MX_ERR_SHAPE, run, **bad)
    refused(api.MX_ERR_FORMAT, run, q=t(3, 4, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        run()
