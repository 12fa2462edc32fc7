"""ctypes binding of libmxgemm.so (declared in include/mxgemm.h).

Argument marshalling only: every entry point has the C name, takes torch tensors (or raw integer
pointers) and an optional stream, checks nothing beyond what it needs to marshal, and raises
MXError when the library returns a non-zero status. All arithmetic runs in the HIP library; if
the shared library is missing this module raises at import time.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmxgemm.so")

MX_E4M3, MX_E5M2, MX_E2M3, MX_E3M2, MX_E2M1, MX_E8M0, MX_F16, MX_INT8, MX_INT4 = 0, 1, 2, 3, 4, 8, 16, 32, 33
MX_BF16, MX_F32 = 17, 18  # rotary positions and the key-value cache only
MXGEMM_RELU = 1  # mxgemm_create flag: C = max(A*B, 0) in the epilogue
MXGEMM_QUANT_A = 2  # mxgemm_create flag: A is binary16, quantised to E4M3 inside the GEMM
MX_OK, MX_ERR_NULL, MX_ERR_SHAPE, MX_ERR_ALIGN, MX_ERR_FORMAT, MX_ERR_ARCH, MX_ERR_LAUNCH, MX_ERR_NOMEM = \
    0, -1, -2, -3, -4, -5, -6, -7
MX_ERR_SCRATCH = -8
MXROPE_HALF, MXROPE_PAIRS = 0, 1  # which elements a rotation pairs
MXROPE_PLAIN, MXROPE_LINEAR, MXROPE_NTK, MXROPE_BANDS, MXROPE_YARN = range(5)  # frequency rules
MXKV_HEADS_FIRST, MXKV_SLOTS_FIRST = 0, 1  # order of a page's elements
MXMATVEC_SCRATCH_BYTES = 17 << 20  # static scratch of mxmatvec_run_noalloc, per GPU

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m block_scaled_quantized_amd.build`")



def _load_hip() -> None:
    """Load torch's own copy of the HIP runtime before the library asks for one. torch needs that copy under a name by which
    the loader does not find a runtime that is loaded already, so a process that loaded the library first
    and torch later had two, and the library's saw no device. (Without torch, the system's is loaded.)"""
    import importlib.util
    import sys
    if "torch" in sys.modules:
        return
    spec = importlib.util.find_spec("torch")
    for home in (spec.submodule_search_locations or []) if spec else []:
        path = os.path.join(home, "lib", "libamdhip64.so")
        if os.path.exists(path):
            ctypes.CDLL(path)
            return


_load_hip()
_lib = ctypes.CDLL(LIB_PATH)
_vp, _i, _u, _i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_int64

_pi = ctypes.POINTER(_i)


class _Heads(ctypes.Structure):
    _fields_ = [("data", _vp), ("heads", _i), ("token_stride", _i64), ("head_stride", _i64)]


class _Rope(ctypes.Structure):
    _fields_ = [("rot_dim", _i), ("layout", _i), ("freq", _vp), ("factor", ctypes.c_float)]


class _Cache(ctypes.Structure):
    _fields_ = [("fmt", _i), ("order", _i), ("pages", _i), ("page_size", _i), ("heads", _i), ("dim", _i),
                ("page_stride", _i64), ("k", _vp), ("v", _vp), ("ks", _vp), ("vs", _vp)]


class _Table(ctypes.Structure):
    _fields_ = [("pages", _vp), ("seqs", _i), ("cols", _i)]


class _AttnOpts(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", _i)]


EXPORTS = {
    "mx_strerror": (ctypes.c_char_p, [_i]),
    "mx_version": (_i, []),
    "mxgemm_create": (_i, [ctypes.POINTER(_vp), _i, _i, _i, _i, _i, _u]),
    "mxgemm_run": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "mxgemm_destroy": (_i, [_vp]),
    "mxgemm_plan_info": (_i, [_vp, ctypes.POINTER(_i), ctypes.POINTER(_i), ctypes.POINTER(_i), ctypes.POINTER(_i)]),
    "mxmatvec_run": (_i, [_i, _i, _i, _vp, _vp, _i, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "mxmatvec_workspace_size": (ctypes.c_size_t, [_i, _i, _i, _i]),
    "mxmatvec_run_noalloc": (_i, [_i, _i, _i, _vp, _vp, _i, _vp, _vp, _vp]),
    "mx_pack_run": (_i, [_i, _vp, _i, _i, _vp, _vp, _vp]),
    "mx_unpack_run": (_i, [_i, _vp, _vp, _i, _i, _vp, _vp]),
    "mxrope_freqs_host": (_i, [_i, ctypes.c_double, _i, _vp, _vp, _vp]),
    "mxrope_run": (_i, [_i, _vp, _i, _i, _vp, _vp, _vp, _i, _vp]),
    "mxkv_append_run": (_i, [_vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "mxattn_decode_run": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, ctypes.c_size_t, _vp]),
    "mxattn_decode_workspace_size": (ctypes.c_size_t, [_vp, _i, _i, _i, _i]),
    "mxkv_copy_run": (_i, [_vp, _i, _vp, _i, _vp]),
    "mxkv_pool_create": (_i, [ctypes.POINTER(_vp), _i, _i, _i, _i]),
    "mxkv_pool_destroy": (_i, [_vp]),
    "mxkv_pool_resize": (_i, [_vp, _i, _i, _vp, _pi]),
    "mxkv_pool_fork": (_i, [_vp, _i, _i]),
    "mxkv_pool_reorder": (_i, [_vp, _vp]),
    "mxkv_pool_compact": (_i, [_vp, _vp, _i, _pi]),
    "mxkv_pool_table": (_vp, [_vp]),
    "mxkv_pool_lengths": (_vp, [_vp]),
    "mxkv_pool_used": (_i, [_vp]),
    "mx_pack_host": (_i, [_i, _vp, _i64, _i64, _vp, _vp]),
    "mx_unpack_host": (_i, [_i, _vp, _vp, _i64, _i64, _vp]),
    "mx_encode_host": (ctypes.c_uint8, [_i, ctypes.c_float]),
    "mx_decode_host": (ctypes.c_float, [_i, ctypes.c_uint8]),
}
for _name, (_res, _args) in EXPORTS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class MXError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {mx_strerror(status)} (status {status})")


def _check(status: int, where: str) -> None:
    if status != MX_OK:
        raise MXError(status, where)


def _ptr(t) -> int | None:
    """Device/host address of a tensor or ndarray, or an int passed through (None stays None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    return t.ctypes.data  # numpy


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def mx_strerror(status: int) -> str:
    return _lib.mx_strerror(status).decode()


def mx_version() -> int:
    return _lib.mx_version()


class Plan:
    """Owns an mxgemm_t; released by mxgemm_destroy when garbage-collected or on close()."""

    def __init__(self, handle: int, M: int, N: int, K: int, fa: int, fb: int):
        self.handle, self.M, self.N, self.K, self.fa, self.fb = handle, M, N, K, fa, fb

    def close(self):
        if self.handle:
            _lib.mxgemm_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def mxgemm_create(M: int, N: int, K: int, fa: int, fb: int, flags: int = 0) -> Plan:
    h = _vp()
    _check(_lib.mxgemm_create(ctypes.byref(h), M, N, K, fa, fb, flags), "mxgemm_create")
    return Plan(h.value, M, N, K, fa, fb)


def mxgemm_plan_info(plan: Plan):
    """(tile_m, tile_n, tile_k, variant) of the kernel chosen by the plan."""
    a, b, c, v = _i(), _i(), _i(), _i()
    _check(_lib.mxgemm_plan_info(plan.handle, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c), ctypes.byref(v)),
           "mxgemm_plan_info")
    return a.value, b.value, c.value, v.value


def mxgemm_run(plan: Plan, A, SA, B, SB, C, stream=None) -> None:
    _check(_lib.mxgemm_run(plan.handle, _ptr(A), _ptr(SA), _ptr(B), _ptr(SB), _ptr(C), _stream(stream)), "mxgemm_run")


def mxgemm_destroy(plan: Plan) -> None:
    plan.close()


def mxmatvec_run(M: int, N: int, K: int, x, W, fw: int, Ws, y, workspace=None, workspace_bytes=None,
                 stream=None) -> None:
    """workspace: a zero-filled device buffer (tensor or address) of workspace_bytes bytes (a
    tensor's own size when omitted), or None for the single-pass kernel."""
    if workspace is not None and workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(_lib.mxmatvec_run(M, N, K, _ptr(x), _ptr(W), fw, _ptr(Ws), _ptr(y), _ptr(workspace),
                             int(workspace_bytes or 0), _stream(stream)), "mxmatvec_run")


def mxmatvec_run_noalloc(M: int, N: int, K: int, x, W, fw: int, Ws, y, stream=None) -> None:
    """mxmatvec_run with the library's static scratch array in place of a workspace."""
    _check(_lib.mxmatvec_run_noalloc(M, N, K, _ptr(x), _ptr(W), fw, _ptr(Ws), _ptr(y), _stream(stream)),
           "mxmatvec_run_noalloc")


def mxmatvec_workspace_size(M: int, N: int, K: int, fw: int) -> int:
    return int(_lib.mxmatvec_workspace_size(M, N, K, fw))


def mx_pack_run(f: int, src, rows: int, cols: int, codes, scales, stream=None) -> None:
    _check(_lib.mx_pack_run(f, _ptr(src), rows, cols, _ptr(codes), _ptr(scales), _stream(stream)), "mx_pack_run")


def mx_unpack_run(f: int, codes, scales, rows: int, cols: int, out, stream=None) -> None:
    _check(_lib.mx_unpack_run(f, _ptr(codes), _ptr(scales), rows, cols, _ptr(out), _stream(stream)), "mx_unpack_run")


def mx_pack_host(f: int, src, rows: int, cols: int, codes, scales) -> None:
    _check(_lib.mx_pack_host(f, _ptr(src), rows, cols, _ptr(codes), _ptr(scales)), "mx_pack_host")


def mx_unpack_host(f: int, codes, scales, rows: int, cols: int, out) -> None:
    _check(_lib.mx_unpack_host(f, _ptr(codes), _ptr(scales), rows, cols, _ptr(out)), "mx_unpack_host")


def mx_encode_host(f: int, v: float) -> int:
    return int(_lib.mx_encode_host(f, v))


def mx_decode_host(f: int, code: int) -> float:
    return float(_lib.mx_decode_host(f, code))


# ---- allocation helpers (torch for device memory; sizes follow the layouts in mxgemm.h) --------

def mx_shapes(fmt: int, rows: int, K: int):
    """(codes shape, scales shape) of an MX operand with `rows` rows of K elements."""
    if fmt == MX_E2M1:
        codes = (rows, K // 2)
    elif fmt in (MX_E2M3, MX_E3M2):
        codes = (rows, K // 4 * 3)
    else:
        codes = (rows, K)
    return codes, (rows, K // 32)


def int_shapes(fw: int, K: int, N: int):
    """(codes shape, scales shape) of an int8/int4 weight W[K][N]."""
    return ((K, N // 2) if fw == MX_INT4 else (K, N)), (K // 32, N)


# ---- the decode step's cache: rotary positions, append, attention, pages ------------------------

def _ints(where: str, *values) -> None:
    """Refuses numbers that ctypes would cut to their low 32 bits."""
    if not all(-1 << 31 <= v < 1 << 31 for v in values):
        raise MXError(MX_ERR_SHAPE, where)


def _on_host(*tensors) -> bool:
    """Whether one of these is a tensor or array in host memory that the GPU cannot read."""
    return any(t is not None and not isinstance(t, int) and not (hasattr(t, "data_ptr") and (t.is_cuda or t.numel() == 0 or t.is_pinned())) for t in tensors)


class Rope:
    """An mxrope: freq is a device tensor of rot_dim / 2 doubles (or more), which is kept alive here, or an address."""

    def __init__(self, rot_dim: int, freq, layout: int = MXROPE_HALF, factor: float = 1.0):
        _ints("Rope", rot_dim)
        if hasattr(freq, "data_ptr"):
            if not freq.dtype.is_floating_point or freq.element_size() != 8:
                raise MXError(MX_ERR_FORMAT, "Rope")
            if not freq.is_contiguous() or freq.numel() < rot_dim // 2:
                raise MXError(MX_ERR_SHAPE, "Rope")
        self.freq, self.host = freq, _on_host(freq)
        self.c = _Rope(rot_dim, layout, _ptr(freq), factor)
        self.ref = ctypes.addressof(self.c)


def mxrope_freqs_host(rot_dim: int, base: float, rule: int = MXROPE_PLAIN, params=()):
    """(list of rot_dim / 2 angles per position, factor of cos and sin) of a frequency rule."""
    _ints("mxrope_freqs_host", rot_dim, rule)
    freq, factor = (ctypes.c_double * max(1, rot_dim // 2))(), ctypes.c_float()
    par = (ctypes.c_double * 4)(*params) if len(params) else None
    _check(_lib.mxrope_freqs_host(rot_dim, base, rule, par, freq, ctypes.addressof(factor)), "mxrope_freqs_host")
    return list(freq), factor.value


_marshal = None


def _load():
    """The module that turns tensors into descriptors for the calls below (csrc/marshal.cpp); it needs torch."""
    global _marshal
    import torch  # noqa: F401  (loads the libraries that the module is linked to)
    try:
        from . import _marshal as m
    except ImportError as e:
        raise ImportError(f"the module _marshal.so is missing or does not load: build it with `python -m block_scaled_quantized_amd.build`, with torch installed ({e})") from e
    _marshal = m
    return m


def mxrope_run(f: int, rope: Rope, x, out, positions, inverse: bool = False, stream=None) -> None:
    """x, out: [tokens][heads][dim] (out may be x); positions: int32 [tokens]."""
    s = (_marshal or _load()).rope(f, rope.ref, x, out, positions, inverse, None if stream is None else _stream(stream), rope.host)
    if s:
        raise MXError(s, "mxrope_run")


class KVCache:
    """An mxkv_cache over torch tensors, which are kept alive here: k and v are
    [pages][heads][page_size][dim] (MXKV_HEADS_FIRST) or [pages][page_size][heads][dim]
    (MXKV_SLOTS_FIRST), dense within a page; for MX_E4M3 bytes, with the scales ks, vs
    [pages][..][..][dim / 32]. Their types are the format's, or whole numbers of its size that stand for the bits."""

    def __init__(self, fmt: int, k, v, ks=None, vs=None, order: int = MXKV_HEADS_FIRST):
        pages, a, b, dim = k.shape
        stride = k.stride(0) if pages > 1 else a * b * dim
        for t, d, unit in ((k, dim, 1), (v, dim, 1), (ks, dim // 32, 32), (vs, dim // 32, 32)):
            if t is None:
                continue
            if tuple(t.shape) != (pages, a, b, d) or not t[0].is_contiguous() or (pages > 1 and t.stride(0) * unit != stride):
                raise MXError(MX_ERR_SHAPE, "KVCache")
        plane = {MX_F16: "float16", MX_BF16: "bfloat16", MX_E4M3: "float8_e4m3fn"}.get(fmt)
        for t, size, kind in ((k, 1 if fmt == MX_E4M3 else 2, plane), (v, 1 if fmt == MX_E4M3 else 2, plane), (ks, 1, "float8_e8m0fnu"), (vs, 1, "float8_e8m0fnu")):
            if t is not None and (t.element_size() != size or (t.dtype.is_floating_point and str(t.dtype) != f"torch.{kind}")):
                raise MXError(MX_ERR_FORMAT, "KVCache")
        heads, page_size = (a, b) if order == MXKV_HEADS_FIRST else (b, a)
        self.tensors, self.host = (k, v, ks, vs), _on_host(k, v, ks, vs)
        self.c = _Cache(fmt, order, pages, page_size, heads, dim, stride, _ptr(k), _ptr(v), _ptr(ks), _ptr(vs))
        self.ref = ctypes.addressof(self.c)


def kv_layers(caches):
    """The layers' caches as the array that mxkv_copy_run takes, for callers that keep it."""
    arr = (_Cache * max(1, len(caches)))(*(x.c for x in caches))
    arr.count, arr.caches, arr.host = len(caches), list(caches), any(x.host for x in caches)
    return arr


def mxkv_append_run(cache: KVCache, f: int, k, v, positions, table, seq=None, rope: Rope | None = None, q=None, q_out=None,
                    stream=None) -> None:
    """k, v: [tokens][heads][dim]; positions, seq: int32 [tokens]; table: int32 [seqs][cols]; q, q_out:
    [tokens][q heads][dim], turned in the same launch."""
    s = (_marshal or _load()).append(cache.ref, f, k, v, positions, table, seq, rope.ref if rope else None, q, q_out,
                                     None if stream is None else _stream(stream), cache.host or (rope is not None and rope.host))
    if s:
        raise MXError(s, "mxkv_append_run")


def mxattn_decode_workspace_size(cache: KVCache, seqs: int, q_heads: int, max_len: int, window: int = 0) -> int:
    _ints("mxattn_decode_workspace_size", seqs, q_heads, max_len, window)
    return int(_lib.mxattn_decode_workspace_size(cache.ref, seqs, q_heads, max_len, window))


def mxattn_decode_run(cache: KVCache, f: int, q, out, table, lengths, max_len: int, scale: float, lse=None, starts=None,
                      window: int = 0, softcap: float = 0.0, workspace=None, workspace_bytes=None, stream=None) -> None:
    """q, out: [seqs][q heads][dim]; table: int32 [seqs][cols]; lengths, starts: int32 [seqs]; lse: fp32
    [seqs][q heads]; workspace: a zero-filled device buffer (a tensor's own size when workspace_bytes is omitted)."""
    s = (_marshal or _load()).attention(cache.ref, f, q, out, table, lengths, max_len, scale, lse, starts, window, softcap,
                                        workspace, workspace_bytes, None if stream is None else _stream(stream), cache.host)
    if s:
        raise MXError(s, "mxattn_decode_run")


def mxkv_copy_run(caches, pairs, stream=None) -> None:
    """caches: a list of KVCache, or kv_layers of it; pairs: int32 [n][2] of (source, destination) pages."""
    arr = caches if isinstance(caches, ctypes.Array) else kv_layers(caches)
    s = (_marshal or _load()).copy(ctypes.addressof(arr), arr.count, pairs, None if stream is None else _stream(stream), arr.host)
    if s:
        raise MXError(s, "mxkv_copy_run")


class KVPool:
    """Owns an mxkv_pool. Page pairs come back as lists of (source, destination) for mxkv_copy_run."""

    def __init__(self, pages: int, page_size: int, seqs: int, cols: int):
        h = _vp()
        self.handle = None
        _ints("mxkv_pool_create", pages, page_size, seqs, cols)
        _check(_lib.mxkv_pool_create(ctypes.byref(h), pages, page_size, seqs, cols), "mxkv_pool_create")
        self.handle, self.pages, self.seqs, self.cols = h.value, pages, seqs, cols

    def close(self):
        if self.handle:
            _lib.mxkv_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def resize(self, seq: int, tokens: int):
        _ints("mxkv_pool_resize", seq, tokens)
        pair, n = (ctypes.c_int32 * 2)(), _i()
        _check(_lib.mxkv_pool_resize(self.handle, seq, tokens, pair, ctypes.byref(n)), "mxkv_pool_resize")
        return [(pair[0], pair[1])] if n.value else []

    def fork(self, src: int, dst: int) -> None:
        _ints("mxkv_pool_fork", src, dst)
        _check(_lib.mxkv_pool_fork(self.handle, src, dst), "mxkv_pool_fork")

    def reorder(self, source) -> None:
        if len(source) != self.seqs:
            raise MXError(MX_ERR_SHAPE, "mxkv_pool_reorder")
        _ints("mxkv_pool_reorder", *source)
        _check(_lib.mxkv_pool_reorder(self.handle, (ctypes.c_int32 * self.seqs)(*source)), "mxkv_pool_reorder")

    def compact(self, max_pairs: int | None = None):
        most = self.pages if max_pairs is None else max_pairs
        _ints("mxkv_pool_compact", most)
        pairs, n = (ctypes.c_int32 * max(1, 2 * most))(), _i()
        _check(_lib.mxkv_pool_compact(self.handle, pairs, most, ctypes.byref(n)), "mxkv_pool_compact")
        return [(pairs[2 * i], pairs[2 * i + 1]) for i in range(n.value)]

    def _host(self, name, shape):
        import numpy as np
        at = getattr(_lib, name)(self.handle)
        return np.ctypeslib.as_array(ctypes.cast(at, ctypes.POINTER(ctypes.c_int32)), shape).copy()

    def table(self):
        """numpy int32 [seqs][cols], -1 where a sequence has no page."""
        return self._host("mxkv_pool_table", (self.seqs, self.cols))

    def lengths(self):
        return self._host("mxkv_pool_lengths", (self.seqs,))

    @property
    def used(self) -> int:
        return _lib.mxkv_pool_used(self.handle)
