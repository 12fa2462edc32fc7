"""Host side of the decode step's cache: frequency rules, refusals of every entry point (no GPU work is
queued) and the page pool against a plain model."""
import ctypes
import math
import random

import numpy as np
import pytest

api = pytest.importorskip("block_scaled_quantized_amd.api")
lib = api._lib


# ---- frequency rules ----------------------------------------------------------------------------

@pytest.mark.parametrize("rot", [2, 20, 64, 128, 256])
@pytest.mark.parametrize("rule,params", [("plain", ()), ("linear", (4.0,)), ("ntk", (8.0,)), ("bands", (8.0, 8192.0, 1.0, 4.0)),
                                         ("yarn", (16.0, 4096.0, 32.0, 1.0))])
def test_frequencies(rot, rule, params):
    base = 10000.0
    got, factor = api.mxrope_freqs_host(rot, base, getattr(api, "MXROPE_" + rule.upper()), params)
    want = []
    for i in range(rot // 2):
        b = base * params[0] ** (rot / (rot - 2)) if rule == "ntk" and rot > 2 else base
        f = b ** (-2 * i / rot)
        if rule == "linear":
            f /= params[0]
        elif rule == "bands":
            turns = params[1] * f / (2 * math.pi)
            k = min(max((turns - params[2]) / (params[3] - params[2]), 0), 1)
            f = (1 - k) * f / params[0] + k * f
        elif rule == "yarn":
            index = [rot * math.log(params[1] / (t * 2 * math.pi)) / (2 * math.log(base)) for t in params[2:]]
            a, c = max(math.floor(index[0]), 0), min(math.ceil(index[1]), rot - 1)
            r = min(max((i - a) / max(c - a, 0.001), 0), 1)
            f = r * f / params[0] + (1 - r) * f
        want.append(f)
    assert len(got) == rot // 2
    np.testing.assert_allclose(got, want, rtol=16 * 2.0 ** -53 * 64, atol=0)
    assert factor == np.float32(0.1 * math.log(16.0) + 1 if rule == "yarn" else 1.0)


@pytest.mark.parametrize("args,status", [
    ((3, 1e4, 0, None), "SHAPE"), ((0, 1e4, 0, None), "SHAPE"), ((258, 1e4, 0, None), "SHAPE"), ((64, 0.0, 0, None), "SHAPE"),
    ((64, math.inf, 0, None), "SHAPE"), ((64, math.nan, 0, None), "SHAPE"), ((64, 1e4, 5, None), "FORMAT"), ((64, 1e4, -1, None), "FORMAT"),
    ((64, 1e4, 1, None), "NULL"), ((64, 1e4, 1, (0.0,)), "SHAPE"), ((64, 1e4, 2, (-1.0,)), "SHAPE"), ((64, 1e4, 1, (math.nan,)), "SHAPE"),
    ((64, 1e4, 3, (8.0, 8192.0, 4.0, 4.0)), "SHAPE"), ((64, 1e4, 3, (8.0, 0.0, 1.0, 4.0)), "SHAPE"),
    ((64, 1.0, 4, (8.0, 4096.0, 32.0, 1.0)), "SHAPE"), ((64, 1e4, 4, (8.0, 4096.0, 0.0, 1.0)), "SHAPE")])
def test_frequency_refusals(args, status):
    rot, base, rule, params = args
    freq, factor = (ctypes.c_double * 128)(*([7.0] * 128)), ctypes.c_float(7.0)
    par = (ctypes.c_double * 4)(*params) if params else None
    assert lib.mxrope_freqs_host(rot, base, rule, par, freq, ctypes.addressof(factor)) == getattr(api, "MX_ERR_" + status)
    assert set(freq) == {7.0} and factor.value == 7.0
    assert lib.mxrope_freqs_host(64, 1e4, 0, None, None, ctypes.addressof(factor)) == api.MX_ERR_NULL


# ---- refusals: addresses are never followed, so any aligned number stands for device memory ------

P = 1 << 20


def heads(data=P, n=8, token=8 * 128, head=128):
    return api._Heads(data, n, token, head)


def cache(**kw):
    c = dict(fmt=api.MX_E4M3, order=0, pages=16, page_size=16, heads=8, dim=128, page_stride=16 * 8 * 128, k=P, v=2 * P, ks=3 * P, vs=4 * P)
    c.update(kw)
    return api._Cache(*[c[n] for n, _ in api._Cache._fields_])


def at(x):
    return ctypes.byref(x) if isinstance(x, (ctypes.Structure, ctypes.Array)) else x


def rope(rot=128, layout=0, freq=P):
    return api._Rope(rot, layout, freq, 1.0)


BAD_HEADS = [(dict(data=None), "NULL"), (dict(data=P + 8), "ALIGN"), (dict(n=0), "SHAPE"), (dict(token=1020), "SHAPE"), (dict(head=129), "SHAPE")]
BAD_ROPE = [(dict(freq=None), "NULL"), (dict(freq=P + 4), "ALIGN"), (dict(rot=0), "SHAPE"), (dict(rot=63), "SHAPE"), (dict(rot=130), "SHAPE"),
            (dict(layout=2), "FORMAT")]
BAD_CACHE = [(dict(fmt=api.MX_E5M2), "FORMAT"), (dict(fmt=api.MX_F32), "FORMAT"), (dict(order=2), "FORMAT"), (dict(pages=0), "SHAPE"),
             (dict(page_size=0), "SHAPE"), (dict(pages=1 << 27), "SHAPE"), (dict(heads=0), "SHAPE"), (dict(heads=1025), "SHAPE"),
             (dict(dim=0), "SHAPE"), (dict(dim=120), "SHAPE"), (dict(dim=288), "SHAPE"), (dict(page_stride=16 * 8 * 128 - 32), "SHAPE"),
             (dict(page_stride=16 * 8 * 128 + 16), "SHAPE"), (dict(k=None), "NULL"), (dict(vs=None), "NULL"), (dict(v=P + 4), "ALIGN"),
             (dict(ks=P + 1), "ALIGN")]


def run_rope(f=api.MX_F16, r=None, tokens=4, dim=128, x=None, out=None, pos=P):
    return lib.mxrope_run(f, at(r or rope()), tokens, dim, at(x or heads()), at(out or heads(2 * P)), pos, 0, None)


def test_rope_refusals():
    for kw, s in BAD_ROPE:
        assert run_rope(r=rope(**kw)) == getattr(api, "MX_ERR_" + s), kw
    for kw, s in BAD_HEADS:
        assert run_rope(x=heads(**kw)) == getattr(api, "MX_ERR_" + s), kw
        assert run_rope(out=heads(**kw)) == getattr(api, "MX_ERR_" + s), kw
    assert run_rope(f=api.MX_E4M3) == api.MX_ERR_FORMAT
    assert run_rope(f=api.MX_INT8) == api.MX_ERR_FORMAT
    for kw in (dict(tokens=-1), dict(tokens=(1 << 20) + 1), dict(dim=4), dict(dim=264), dict(dim=100), dict(out=heads(2 * P, n=4)),
               dict(x=heads(n=65537), out=heads(2 * P, n=65537)), dict(out=heads(P, token=2048))):
        assert run_rope(**kw) == api.MX_ERR_SHAPE, kw
    assert run_rope(pos=None) == api.MX_ERR_NULL
    assert lib.mxrope_run(api.MX_F16, None, 4, 128, at(heads()), at(heads()), P, 0, None) == api.MX_ERR_NULL
    assert lib.mxrope_run(api.MX_F16, at(rope()), 4, 128, None, at(heads()), P, 0, None) == api.MX_ERR_NULL
    assert run_rope(tokens=0, pos=None, x=heads(None), out=heads(None)) == api.MX_OK   # an empty call needs no memory


def run_append(c=None, f=api.MX_F16, tokens=4, k=None, v=None, pos=P, seq=None, table=None, r=None, q=None, q_out=None):
    return lib.mxkv_append_run(at(c or cache()), f, tokens, at(k or heads()), at(v or heads(2 * P)), pos, seq,
                               at(table or api._Table(P, 4, 8)), at(r), at(q), at(q_out), None)


def test_append_refusals():
    for kw, s in BAD_CACHE:
        assert run_append(c=cache(**kw)) == getattr(api, "MX_ERR_" + s), kw
    for kw, s in BAD_HEADS:
        assert run_append(k=heads(**kw)) == getattr(api, "MX_ERR_" + s), kw
        assert run_append(v=heads(**kw)) == getattr(api, "MX_ERR_" + s), kw
        assert run_append(r=rope(), q=heads(**kw), q_out=heads()) == getattr(api, "MX_ERR_" + s), kw
        assert run_append(r=rope(), q=heads(5 * P), q_out=heads(**kw)) == getattr(api, "MX_ERR_" + s), kw
    for kw, s in BAD_ROPE:
        assert run_append(r=rope(**kw)) == getattr(api, "MX_ERR_" + s), kw
    for f in (api.MX_F32, api.MX_E4M3):
        assert run_append(f=f) == api.MX_ERR_FORMAT
    assert run_append(c=cache(fmt=api.MX_BF16, ks=None, vs=None)) == api.MX_ERR_FORMAT      # fp16 into a bf16 cache
    for kw in (dict(tokens=-1), dict(k=heads(n=4)), dict(v=heads(n=16)), dict(table=api._Table(P, -1, 8)), dict(table=api._Table(P, 4, 0)),
               dict(r=rope(), q=heads(5 * P, n=16), q_out=heads(6 * P))):
        assert run_append(**kw) == api.MX_ERR_SHAPE, kw
    for kw in (dict(pos=None), dict(table=api._Table(None, 4, 8)), dict(r=rope(), q=heads()), dict(r=rope(), q_out=heads()),
               dict(q=heads(), q_out=heads())):
        assert run_append(**kw) == api.MX_ERR_NULL, kw
    assert run_append(tokens=0, pos=None) == api.MX_OK


def run_attn(c=None, f=api.MX_F16, q=None, out=None, table=None, lengths=P, max_len=64, opts=None, ws=None, ws_bytes=0):
    return lib.mxattn_decode_run(at(c or cache()), f, at(q or heads(n=32)), at(out or heads(2 * P, n=32)), None,
                                 at(table or api._Table(P, 4, 8)), lengths, None, max_len, at(opts or api._AttnOpts(1.0, 0.0, 0)), ws, ws_bytes, None)


def test_attention_refusals():
    for kw, s in BAD_CACHE:
        assert run_attn(c=cache(**kw)) == getattr(api, "MX_ERR_" + s), kw
    for kw, s in BAD_HEADS:
        assert run_attn(q=heads(**dict(dict(n=32), **kw)), out=heads(n=kw.get("n", 32))) == getattr(api, "MX_ERR_" + s), kw
        assert run_attn(out=heads(**dict(dict(n=32), **kw))) == getattr(api, "MX_ERR_" + s), kw
    assert run_attn(f=api.MX_F32) == api.MX_ERR_FORMAT
    assert run_attn(c=cache(fmt=api.MX_F16), f=api.MX_BF16) == api.MX_ERR_FORMAT
    opts = api._AttnOpts
    for kw in (dict(q=heads(n=12), out=heads(n=12)), dict(max_len=0), dict(max_len=1 << 30), dict(opts=opts(math.nan, 0.0, 0)),
               dict(opts=opts(1.0, -1.0, 0)), dict(opts=opts(1.0, math.inf, 0)), dict(opts=opts(1.0, 0.0, -1)), dict(table=api._Table(P, -1, 8)),
               dict(table=api._Table(P, 1 << 20, 8))):
        assert run_attn(**kw) == api.MX_ERR_SHAPE, kw
    assert run_attn(lengths=None) == api.MX_ERR_NULL
    assert run_attn(table=api._Table(None, 4, 8)) == api.MX_ERR_NULL
    assert run_attn(ws=P + 8, ws_bytes=1 << 20) == api.MX_ERR_ALIGN
    assert run_attn(table=api._Table(None, 0, 8), lengths=None) == api.MX_OK


def test_attention_workspace_size():
    def size(seqs, q_heads, max_len, window=0, **kw):
        return lib.mxattn_decode_workspace_size(at(cache(**kw)), seqs, q_heads, max_len, window)
    assert size(1, 32, 128) == 0 and size(0, 32, 4096) == 0 and size(1, 12, 4096) == 0 and size(1, 32, 4096, dim=100) == 0
    assert size(1, 32, 1 << 17) > size(1, 32, 4096) > 0
    assert lib.mxattn_decode_workspace_size(None, 1, 32, 4096, 0) == 0
    for seqs in (1, 3, 40, 1000):                 # a workspace for the longest row serves every window
        full = size(seqs, 32, 40000)
        assert all(size(seqs, 32, 40000, w) <= full for w in range(1, 40000, 997))


def test_copy_refusals():
    def run(layers, n_layers=None, pairs=P, n=3):
        arr = (api._Cache * max(1, len(layers)))(*layers)
        return lib.mxkv_copy_run(at(arr), len(layers) if n_layers is None else n_layers, pairs, n, None)
    for kw, s in BAD_CACHE:
        assert run([cache(), cache(**kw)]) in (getattr(api, "MX_ERR_" + s),), kw
    for kw in (dict(order=1), dict(pages=15), dict(page_stride=16 * 8 * 128 + 32), dict(fmt=api.MX_F16), dict(dim=96), dict(heads=4),
               dict(page_size=8)):
        assert run([cache(), cache(**kw)]) == api.MX_ERR_SHAPE, kw
    assert run([cache()], n=-1) == api.MX_ERR_SHAPE and run([cache()], n_layers=-1) == api.MX_ERR_SHAPE
    assert run([cache()], pairs=None) == api.MX_ERR_NULL
    assert lib.mxkv_copy_run(None, 1, P, 1, None) == api.MX_ERR_NULL
    assert run([cache()], n=0, pairs=None) == api.MX_OK and run([], pairs=None) == api.MX_OK


def test_no_device_is_an_error():
    import torch
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    assert run_rope() == api.MX_ERR_ARCH
    assert run_append() == api.MX_ERR_ARCH
    assert run_attn() == api.MX_ERR_ARCH
    arr = (api._Cache * 1)(cache())
    assert lib.mxkv_copy_run(at(arr), 1, P, 1, None) == api.MX_ERR_ARCH


def test_python_refusals():
    import torch
    x = torch.zeros(4, 8, 128, dtype=torch.float16)
    r, pos = api.Rope(128, P), torch.zeros(4, dtype=torch.int32)
    for bad in (dict(x=x.transpose(1, 2)), dict(out=x[:2]), dict(positions=pos.long()), dict(positions=pos[:3])):
        kw = dict(x=x, out=x, positions=pos)
        kw.update(bad)
        with pytest.raises(api.MXError) as e:
            api.mxrope_run(api.MX_F16, r, kw["x"], kw["out"], kw["positions"], stream=0)
        assert e.value.status == api.MX_ERR_SHAPE
    k = torch.zeros(5, 2, 16, 64, dtype=torch.float16)
    api.KVCache(api.MX_F16, k, k)
    for bad in (k[:4], k.transpose(1, 2), torch.zeros(5, 2, 16, 32)):
        with pytest.raises(api.MXError):
            api.KVCache(api.MX_F16, k, bad)
    with pytest.raises(api.MXError):
        api.KVCache(api.MX_E4M3, k, k, k[..., :1], k[..., :1])
    both = torch.zeros(5, 2, 2, 16, 64, dtype=torch.float16)           # keys and values in one allocation
    assert api.KVCache(api.MX_F16, both[:, 0], both[:, 1]).c.page_stride == 2 * 2 * 16 * 64


def test_python_refusals_of_the_cache_calls():
    """Shapes and element sizes that do not fit are refused before the library is called; what is no tensor is a
    TypeError."""
    import torch

    def half(*shape):
        return torch.zeros(*shape, dtype=torch.float16)

    def ints(*shape):
        return torch.zeros(*shape, dtype=torch.int32)

    k = half(5, 2, 16, 64)
    c = api.KVCache(api.MX_F16, k, k)
    rope = api.Rope(64, P)
    good = dict(k=half(4, 2, 64), v=half(4, 2, 64), positions=ints(4), table=ints(3, 5), seq=ints(4), rope=rope, q=half(4, 8, 64), q_out=half(4, 8, 64))
    for bad, status in ((dict(k=half(4, 2, 32)), "SHAPE"), (dict(v=half(3, 2, 64)), "SHAPE"), (dict(q=half(3, 8, 64)), "SHAPE"), (dict(q_out=half(4, 8, 64).transpose(1, 2)), "SHAPE"),
                        (dict(positions=ints(5)), "SHAPE"), (dict(seq=ints(4).long()), "SHAPE"), (dict(table=ints(3, 5).t()), "SHAPE"), (dict(table=ints(15)), "SHAPE"),
                        (dict(k=half(4, 2, 64).float()), "FORMAT"), (dict(q_out=half(4, 8, 64).double()), "FORMAT")):
        kw = dict(good, **bad)
        with pytest.raises(api.MXError) as e:
            api.mxkv_append_run(c, api.MX_F16, kw.pop("k"), kw.pop("v"), kw.pop("positions"), kw.pop("table"), stream=0, **kw)
        assert e.value.status == getattr(api, "MX_ERR_" + status), bad
    good = dict(q=half(3, 8, 64), out=half(3, 8, 64), table=ints(3, 5), lengths=ints(3), lse=torch.zeros(3, 8), starts=ints(3))
    for bad, status in ((dict(q=half(3, 8, 32)), "SHAPE"), (dict(out=half(3, 4, 64)), "SHAPE"), (dict(table=ints(4, 5)), "SHAPE"), (dict(lengths=ints(2)), "SHAPE"),
                        (dict(starts=ints(3).short()), "SHAPE"), (dict(lse=torch.zeros(8, 3).t()), "SHAPE"), (dict(lse=torch.zeros(3, 8).half()), "SHAPE"), (dict(lse=torch.zeros(24)), "SHAPE"),
                        (dict(q=half(3, 8, 64).float()), "FORMAT"), (dict(out=half(3, 8, 64).float()), "FORMAT")):
        kw = dict(good, **bad)
        with pytest.raises(api.MXError) as e:
            api.mxattn_decode_run(c, api.MX_F16, kw.pop("q"), kw.pop("out"), kw.pop("table"), kw.pop("lengths"), 80, 0.1, stream=0, **kw)
        assert e.value.status == getattr(api, "MX_ERR_" + status), bad
    for bad in (ints(4), ints(4, 3), ints(4, 2).long(), ints(2, 4).t()):
        with pytest.raises(api.MXError) as e:
            api.mxkv_copy_run([c], bad, stream=0)
        assert e.value.status == api.MX_ERR_SHAPE
    for call in (lambda: api.mxrope_run(api.MX_F16, rope, [1.0], half(1, 1, 64), ints(1), stream=0), lambda: api.mxkv_copy_run([c], 7, stream=0),
                 lambda: api.mxattn_decode_run(c, api.MX_F16, half(3, 8, 64), half(3, 8, 64), ints(3, 5), 3, 80, 0.1, stream=0)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(api.MXError) as e:
        api.mxrope_run(api.MX_F32, rope, half(4, 8, 64), half(4, 8, 64), ints(4), stream=0)
    assert e.value.status == api.MX_ERR_FORMAT
    for args in ((api.MX_F16, k.float(), k.float()), (api.MX_E4M3, k, k, ints(5, 2, 16, 2), ints(5, 2, 16, 2))):
        with pytest.raises(api.MXError) as e:
            api.KVCache(*args)
        assert e.value.status == api.MX_ERR_FORMAT


def test_one_hip_runtime_in_a_process():
    """Whether the package or torch is imported first, both use one copy of the HIP runtime."""
    import subprocess
    import sys
    from conftest import ROOT
    show = "print(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))"
    for first in ("from block_scaled_quantized_amd import api; import torch", "import torch; from block_scaled_quantized_amd import api"):
        r = subprocess.run([sys.executable, "-c", f"{first}; {show}"], cwd=ROOT, capture_output=True, text=True)
        assert r.returncode == 0 and r.stdout.split()[-1] == "1", (first, r.stdout, r.stderr)


# ---- page pool -----------------------------------------------------------------------------------

class Model:
    """The pool's rules, plainly: rows of pages, the lowest free page first."""

    def __init__(self, pages, page, seqs, cols):
        self.n, self.page, self.rows, self.len, self.cols = pages, page, [[] for _ in range(seqs)], [0] * seqs, cols

    def held(self):
        return {p for r in self.rows for p in r}

    def free(self):
        return [p for p in range(self.n) if p not in self.held()]

    def shared(self, p):
        return sum(p in r for r in self.rows) > 1

    def resize(self, s, t):
        row, need, pairs = self.rows[s], -(-t // self.page), []
        own = t > self.len[s] and self.len[s] % self.page and self.shared(row[-1])
        if max(0, need - len(row)) + bool(own) > len(self.free()):
            return None
        if own:
            to = self.free()[0]
            pairs, row[-1] = [(row[-1], to)], to
        while len(row) < need:
            row.append(self.free()[0])
        del row[need:]
        self.len[s] = t
        return pairs

    def compact(self, most):
        pairs, held = [], self.held()
        while len(pairs) < most:
            hole, top = min(set(range(self.n)) - held, default=self.n), max(held, default=-1)
            if hole > top:
                break
            pairs.append((top, hole))
            held = held - {top} | {hole}
            self.rows = [[hole if p == top else p for p in r] for r in self.rows]
        return pairs


@pytest.mark.parametrize("seed", range(6))
def test_pool_follows_the_model(seed):
    r = random.Random(seed)
    pages, page, seqs, cols = r.choice([(7, 4, 3, 4), (40, 1, 6, 9), (64, 16, 9, 12)])
    pool, m = api.KVPool(pages, page, seqs, cols), Model(pages, page, seqs, cols)
    moved = {p: p for p in range(pages)}
    for _ in range(300):
        do = r.random()
        s = r.randrange(seqs)
        if do < 0.6:
            t = r.choice([0, m.len[s] + 1, r.randint(0, cols * page)])
            if t > cols * page:
                continue
            want = m.resize(s, t)
            if want is None:
                with pytest.raises(api.MXError) as e:
                    pool.resize(s, t)
                assert e.value.status == api.MX_ERR_NOMEM
            else:
                assert pool.resize(s, t) == want
        elif do < 0.8:
            d = r.randrange(seqs)
            if s != d and not m.len[d]:
                pool.fork(s, d)
                m.rows[d], m.len[d] = list(m.rows[s]), m.len[s]
            else:
                with pytest.raises(api.MXError):
                    pool.fork(s, d)
        elif do < 0.9:
            order = [r.randrange(seqs) for _ in range(seqs)]
            pool.reorder(order)
            m.rows, m.len = [list(m.rows[i]) for i in order], [m.len[i] for i in order]
        else:
            most = r.choice([0, 1, 3, pages])
            assert pool.compact(most) == m.compact(most)
        assert pool.lengths().tolist() == m.len and pool.used == len(m.held())
        assert pool.table().tolist() == [row + [-1] * (cols - len(row)) for row in m.rows]
    pool.compact()
    assert pool.table().max() < pool.used
    pool.close()


def test_pool_refusals():
    h = ctypes.c_void_p()
    for args in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), ((1 << 20) + 1, 1, 1, 1), (1 << 20, 1 << 20, 1, 1),
                 (1, 1, 1 << 20, 1 << 20), (1, 1 << 20, 1, 1 << 20)):
        assert lib.mxkv_pool_create(ctypes.byref(h), *args) == api.MX_ERR_SHAPE and not h.value, args
    assert lib.mxkv_pool_create(None, 1, 1, 1, 1) == api.MX_ERR_NULL
    pool = api.KVPool(4, 16, 2, 3)
    for seq, t in ((-1, 1), (2, 1), (0, -1), (0, 49)):
        with pytest.raises(api.MXError) as e:
            pool.resize(seq, t)
        assert e.value.status == api.MX_ERR_SHAPE
    assert pool.resize(0, 48) == [] and pool.used == 3
    with pytest.raises(api.MXError) as e:
        pool.resize(1, 32)
    assert e.value.status == api.MX_ERR_NOMEM and pool.used == 3 and pool.lengths().tolist() == [48, 0]
    with pytest.raises(api.MXError):
        pool.reorder([0, 2])
    with pytest.raises(api.MXError):
        pool.reorder([0])
    n, pair = ctypes.c_int(), (ctypes.c_int32 * 2)()
    assert lib.mxkv_pool_resize(None, 0, 1, pair, ctypes.byref(n)) == api.MX_ERR_NULL
    assert lib.mxkv_pool_resize(pool.handle, 0, 1, None, ctypes.byref(n)) == api.MX_ERR_NULL
    assert lib.mxkv_pool_compact(pool.handle, None, 2, ctypes.byref(n)) == api.MX_ERR_NULL
    assert lib.mxkv_pool_compact(pool.handle, pair, -1, ctypes.byref(n)) == api.MX_ERR_SHAPE
    assert lib.mxkv_pool_fork(None, 0, 1) == lib.mxkv_pool_reorder(None, pair) == api.MX_ERR_NULL
    assert lib.mxkv_pool_table(None) is None and lib.mxkv_pool_used(None) == 0 and lib.mxkv_pool_destroy(None) == api.MX_OK


def test_pool_lengths_near_two_to_the_31():
    """A length whose last page ends past 2^31 - 1 when rounded up: its pages are given back, shared and reordered."""
    page, cols = 2049, 1048064
    top = cols * page
    assert top < 2 ** 31 <= top + page - 1
    pool = api.KVPool(cols, page, 2, cols)
    assert pool.resize(0, top) == [] and pool.used == cols
    assert pool.resize(0, 0) == [] and pool.used == 0
    pool.resize(0, top)
    pool.fork(0, 1)
    pool.reorder([1, 1])
    assert pool.used == cols and pool.lengths().tolist() == [top, top] and (pool.table()[1] == pool.table()[0]).all()
    assert pool.compact(4) == []
    pool.resize(0, 0)
    assert pool.used == cols
    pool.resize(1, 0)
    assert pool.used == 0 and (pool.table() == -1).all()
    pool.close()


def test_rope_refuses_frequencies_that_are_not_rot_dim_halves_of_doubles():
    """The kernels read rot_dim / 2 doubles at the tensor's address."""
    import torch
    f = torch.zeros(64, dtype=torch.float64)
    for bad, status in ((f.float(), "FORMAT"), (f.long(), "FORMAT"), (f.half(), "FORMAT"), (f[:63], "SHAPE"), (torch.zeros(128, dtype=torch.float64)[::2], "SHAPE"),
                        (f[:0], "SHAPE"), (torch.zeros(1, dtype=torch.float64).expand(64), "SHAPE")):
        with pytest.raises(api.MXError) as e:
            api.Rope(128, bad)
        assert e.value.status == getattr(api, "MX_ERR_" + status), bad.shape
    for good in (f, torch.zeros(65, dtype=torch.float64), f.reshape(8, 8), P):   # an address stands for itself
        api.Rope(128, good)


def test_python_refuses_tensors_of_another_floating_type():
    """binary16 given as MX_BF16 has the right size and the wrong values; whole-number tensors stand for their bits."""
    import torch

    def x(kind, *shape):
        return torch.zeros(*shape, dtype=kind)

    def ints(*shape):
        return torch.zeros(*shape, dtype=torch.int32)

    half, bf16 = torch.float16, torch.bfloat16
    rope = api.Rope(64, P)
    for f, kind, other in ((api.MX_F16, half, bf16), (api.MX_BF16, bf16, half)):
        for a, b in ((other, kind), (kind, other)):
            with pytest.raises(api.MXError) as e:
                api.mxrope_run(f, rope, x(a, 4, 8, 64), x(b, 4, 8, 64), ints(4), stream=0)
            assert e.value.status == api.MX_ERR_FORMAT
    k = x(half, 5, 2, 16, 64)
    c = api.KVCache(api.MX_F16, k, k)
    for bad in (dict(k=x(bf16, 4, 2, 64)), dict(v=x(bf16, 4, 2, 64)), dict(q=x(bf16, 4, 8, 64)), dict(q_out=x(bf16, 4, 8, 64))):
        kw = dict(dict(k=x(half, 4, 2, 64), v=x(half, 4, 2, 64), q=x(half, 4, 8, 64), q_out=x(half, 4, 8, 64)), **bad)
        with pytest.raises(api.MXError) as e:
            api.mxkv_append_run(c, api.MX_F16, kw["k"], kw["v"], ints(4), ints(3, 5), rope=rope, q=kw["q"], q_out=kw["q_out"], stream=0)
        assert e.value.status == api.MX_ERR_FORMAT, bad
    for q, out in ((bf16, half), (half, bf16)):
        with pytest.raises(api.MXError) as e:
            api.mxattn_decode_run(c, api.MX_F16, x(q, 3, 8, 64), x(out, 3, 8, 64), ints(3, 5), ints(3), 80, 0.1, stream=0)
        assert e.value.status == api.MX_ERR_FORMAT
    codes, scales = x(torch.uint8, 5, 2, 16, 64), x(torch.uint8, 5, 2, 16, 2)
    for args in ((api.MX_BF16, k, k), (api.MX_F16, k, k.bfloat16()), (api.MX_E4M3, codes.view(torch.float8_e5m2), codes, scales, scales),
                 (api.MX_E4M3, codes, codes, scales, scales.view(torch.float8_e4m3fn))):
        with pytest.raises(api.MXError) as e:
            api.KVCache(*args)
        assert e.value.status == api.MX_ERR_FORMAT
    api.KVCache(api.MX_E4M3, codes.view(torch.float8_e4m3fn), codes, scales.view(torch.float8_e8m0fnu), scales)
    api.KVCache(api.MX_BF16, k.view(torch.int16), k.view(torch.int16))


def test_python_refuses_numbers_past_32_bits():
    """Not cut to their low 32 bits: a window of 2^32 is not none, a length of 2^32 + 5 not five."""
    import torch
    q, big = torch.zeros(3, 8, 64, dtype=torch.float16), 1 << 32
    k, n = torch.zeros(5, 2, 16, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    c, table, ws = api.KVCache(api.MX_F16, k, k), torch.zeros(3, 5, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)

    def attend(f=api.MX_F16, max_len=80, **kw):
        return lambda: api.mxattn_decode_run(c, f, q, q, table, n, max_len, 0.1, stream=0, **kw)

    pool = api.KVPool(8, 16, 2, 4)
    pool.resize(0, 5)
    bad = [(attend(f=big + api.MX_F16), "FORMAT"), (attend(max_len=big + 80), "SHAPE"), (attend(max_len=-big + 80), "SHAPE"), (attend(window=big), "SHAPE"),
           (attend(window=big + 7), "SHAPE"), (attend(window=1 << 70), "SHAPE"), (attend(workspace=ws, workspace_bytes=-1), "SHAPE"),
           (attend(workspace=ws, workspace_bytes=65), "SHAPE"), (attend(workspace=ws[::2]), "SHAPE"), (attend(workspace=ws[:1].expand(64)), "SHAPE"),
           (lambda: api.mxrope_run(big + api.MX_F16, api.Rope(64, P), q, q, n, stream=0), "FORMAT"),
           (lambda: api.mxkv_append_run(c, big + api.MX_F16, q[:, :2], q[:, :2], n, table, stream=0), "FORMAT"),
           (lambda: api.Rope(big + 64, P), "SHAPE"), (lambda: api.mxrope_freqs_host(big + 64, 1e4), "SHAPE"),
           (lambda: api.mxattn_decode_workspace_size(c, 3, 8, big + 80), "SHAPE"), (lambda: api.KVPool(8, big + 16, 2, 4), "SHAPE"),
           (lambda: pool.resize(0, big + 7), "SHAPE"), (lambda: pool.resize(big, 7), "SHAPE"), (lambda: pool.fork(0, big + 1), "SHAPE"),
           (lambda: pool.reorder([0, big]), "SHAPE"), (lambda: pool.compact(big + 1), "SHAPE")]
    for i, (call, status) in enumerate(bad):
        with pytest.raises(api.MXError) as e:
            call()
        assert e.value.status == getattr(api, "MX_ERR_" + status), i
    assert pool.lengths().tolist() == [5, 0]


def test_python_refuses_host_tensors():
    """A host tensor's address means nothing to a kernel, which would fault on it: a TypeError once all else is in order."""
    import torch

    def half(*shape):
        return torch.zeros(*shape, dtype=torch.float16)

    def ints(*shape):
        return torch.zeros(*shape, dtype=torch.int32)

    k = half(5, 2, 16, 64)
    c = api.KVCache(api.MX_F16, k, k)
    freq = torch.zeros(32, dtype=torch.float64)
    for call in (lambda: api.mxrope_run(api.MX_F16, api.Rope(64, P), half(4, 8, 64), half(4, 8, 64), ints(4), stream=0),
                 lambda: api.mxrope_run(api.MX_F16, api.Rope(64, freq), half(4, 8, 64), half(4, 8, 64), ints(4), stream=0),
                 lambda: api.mxkv_append_run(c, api.MX_F16, half(4, 2, 64), half(4, 2, 64), ints(4), ints(4, 5), stream=0),
                 lambda: api.mxattn_decode_run(c, api.MX_F16, half(3, 8, 64), half(3, 8, 64), ints(3, 5), ints(3), 80, 0.1, stream=0),
                 lambda: api.mxkv_copy_run([c], ints(4, 2), stream=0), lambda: api.mxkv_copy_run(api.kv_layers([c]), ints(4, 2), stream=0)):
        with pytest.raises(TypeError, match="GPU"):
            call()
    api.mxkv_copy_run([], ints(0, 2), stream=0)                     # nothing is read


@pytest.mark.parametrize("s", [1e-6, 0.25, 0.999, 1.0, 1.5, 16.0])
def test_yarn_factor_is_1_where_nothing_is_stretched(s):
    """The factor makes up for a stretched context: 0.1 ln s + 1 above s = 1, 1 up to it (below 1 otherwise, and negative under
    s = e^-10)."""
    _, factor = api.mxrope_freqs_host(64, 1e4, api.MXROPE_YARN, (s, 4096.0, 32.0, 1.0))
    assert factor == np.float32(0.1 * math.log(s) + 1 if s > 1 else 1.0)


def test_rope_refuses_more_workgroups_than_a_launch_has():
    """Halves that begin within a unit take a workgroup for every 16 KB of rows: 2^20 tokens of 65536 heads of 256 fp32 would be 2^32
    of them, which a 32-bit grid holds as none."""
    rows = dict(n=65536, token=65536 * 256, head=256)
    for tokens, n, status in ((1 << 20, 65536, api.MX_ERR_SHAPE), (1 << 20, 257, api.MX_ERR_SHAPE)):
        x, out = heads(**dict(rows, n=n)), heads(2 * P, **dict(rows, n=n))
        assert run_rope(f=api.MX_F32, r=rope(rot=2), tokens=tokens, dim=256, x=x, out=out) == status


def test_copy_takes_every_number_of_pairs():
    """Up to MX_MAX_DIM pairs, whatever a page's size; a page's plane of 16 GiB and more is refused."""
    import torch

    def run(c, n):
        arr = (api._Cache * 1)(c)
        return lib.mxkv_copy_run(at(arr), 1, P, n, None)
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU: valid calls end at the missing device")
    big = dict(page_size=256, heads=8, dim=128, pages=1 << 16, page_stride=256 * 8 * 128)
    for kw in (dict(fmt=api.MX_F16), dict(fmt=api.MX_E4M3)):
        for n in (1, 1 << 15, 1 << 17, 1 << 20):
            assert run(cache(**big, **kw), n) == api.MX_ERR_ARCH, (kw, n)
    huge = dict(fmt=api.MX_F16, page_size=1 << 20, heads=32, dim=256, pages=2, page_stride=(1 << 20) * 32 * 256)
    assert run(cache(**huge), 1) == api.MX_ERR_SHAPE
    assert run(cache(**dict(huge, heads=31, page_stride=(1 << 20) * 31 * 256)), 7) == api.MX_ERR_ARCH
