"""Cases and plain forms of the decode-time operators: rotary positions, the paged key-value cache's
append, attention of one new token over it, and the copying of its pages.

`run` computes an operator in plain torch operations where `own` is false, and calls this package's
entry points where it is true. Every operator works on the same paged cache: page p of a sequence's
table row holds its positions p * page .. p * page + page - 1, in [pages][heads][page][dim]
("heads") or [pages][page][heads][dim] ("slots") order, as fp16 / bf16 values or as E4M3 codes with
one E8M0 scale per 32 elements of dim.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}

# Rotary scalings: name -> parameters after the base. "bands" and "yarn" are (factor, trained
# length, low, high) and (factor, trained length, fast, slow).
SCALINGS = {"plain": (), "linear": (4.0,), "ntk": (8.0,), "bands": (8.0, 8192.0, 1.0, 4.0), "yarn": (16.0, 4096.0, 32.0, 1.0)}


def listed():
    return [
        # one decoded token of one sequence at a far position: launch latency
        dict(name="rotary one token", op="rotary", tokens=1, heads=32, dim=128, rot=128, layout="half", scaling="bands",
             type="fp16", inverse=False, far=1000000),
        # a prompt's queries, as a slice of the fused projection, with scaled frequencies
        dict(name="rotary prompt", op="rotary", tokens=4096, heads=32, dim=128, rot=128, layout="half", scaling="yarn",
             type="bf16", inverse=False, far=65536),
        # the gradient of a partial, interleaved rotation in full precision (a training step's backward)
        dict(name="rotary backward", op="rotary", tokens=2047, heads=20, dim=80, rot=32, layout="pairs", scaling="plain",
             type="fp32", inverse=True, far=2047),
        # a decode step's keys and values of 64 sequences, rotated and quantised into an E4M3 cache
        dict(name="append decode e4m3", op="append", tokens=64, seqs=64, q_heads=32, heads=8, dim=128, page=64, rot=128,
             layout="half", scaling="plain", type="fp16", cache="e4m3", order="heads", far=4096),
        # ragged prompts written to a bf16 cache of small pages
        dict(name="append prompts bf16", op="append", tokens=8191, seqs=7, q_heads=32, heads=8, dim=128, page=16, rot=128,
             layout="half", scaling="ntk", type="bf16", cache="bf16", order="slots", far=8191),
        # one short sequence: latency
        dict(name="attention short", op="attention", seqs=1, q_heads=32, heads=8, dim=128, page=16, length=500,
             ragged=False, starts=False, window=0, softcap=0.0, type="fp16", cache="fp16", order="heads"),
        # a serving batch of ragged lengths
        dict(name="attention batch ragged", op="attention", seqs=32, q_heads=32, heads=8, dim=128, page=16, length=8192,
             ragged=True, starts=False, window=0, softcap=0.0, type="bf16", cache="bf16", order="slots"),
        # every head its own keys, odd head size and pages, a window, padding on the left, capped scores
        dict(name="attention odd", op="attention", seqs=5, q_heads=12, heads=12, dim=96, page=24, length=3001, ragged=True,
             starts=True, window=1500, softcap=30.0, type="fp16", cache="e4m3", order="slots"),
        # one very long sequence: the length is all there is to split
        dict(name="attention long", op="attention", seqs=1, q_heads=64, heads=8, dim=128, page=64, length=131072,
             ragged=False, starts=False, window=0, softcap=0.0, type="fp16", cache="fp16", order="heads"),
        # a large quantised batch: bandwidth
        dict(name="attention large e4m3", op="attention", seqs=64, q_heads=64, heads=8, dim=128, page=64, length=16384,
             ragged=False, starts=False, window=0, softcap=0.0, type="bf16", cache="e4m3", order="heads"),
        # the last, shared pages of four forked sequences, over eight layers
        dict(name="copy fork", op="copy", layers=8, pages=64, pairs=4, heads=8, dim=128, page=16, cache="bf16",
             order="heads"),
        # a cache's compaction: its high pages move into the holes, over four layers
        dict(name="copy compaction e4m3", op="copy", layers=4, pages=2048, pairs=700, heads=8, dim=128, page=64,
             cache="e4m3", order="slots"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _rotary(rng, dim):
    rot = dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2)
    return dict(rot=rot, layout=rng.choice(["half", "pairs"]), scaling=rng.choice(sorted(SCALINGS)))


def _heads(rng):
    heads = rng.choice([1, 2, 3, 4, 8, 12, 16])
    return heads, heads * rng.choice([1, 2, 4, 5, 7, 8, 16, 20])


def draw(rng):
    op = rng.choice(["rotary", "append", "attention", "attention", "attention", "copy"])
    order = rng.choice(["heads", "slots"])
    kind = rng.choice(["fp16", "bf16"])
    cache = rng.choice([kind, "e4m3"])
    page = rng.choice([16, 32, 64, 128, 256, rng.randint(1, 100)])
    if op == "rotary":
        dim, heads = 8 * rng.randint(1, 32), rng.randint(1, 64)
        return dict(op=op, tokens=_log(rng, 1, min(16384, (1 << 26) // (dim * heads))), heads=heads, dim=dim, **_rotary(rng, dim),
                    type=rng.choice(["fp16", "bf16", "fp32"]), inverse=rng.random() < 0.5, far=_log(rng, 1, 1 << 20))
    if op == "append":
        dim = 32 * rng.randint(1, 8) if cache == "e4m3" else 8 * rng.randint(1, 32)
        heads, q_heads = _heads(rng)
        tokens = _log(rng, 1, min(16384, (1 << 25) // (dim * q_heads)))
        seqs = min(tokens, _log(rng, 1, 256))
        return dict(op=op, tokens=tokens, seqs=seqs, q_heads=q_heads, heads=heads, dim=dim, page=page, **_rotary(rng, dim), type=kind,
                    cache=cache, order=order, far=_log(rng, 1, 32768))
    if op == "copy":
        dim = 32 * rng.randint(1, 8) if cache == "e4m3" else 8 * rng.randint(1, 32)
        heads, layers = rng.choice([1, 2, 4, 8, 16]), _log(rng, 1, 40)
        most = (1 << 29) // (layers * heads * dim * page)
        pages = _log(rng, 2, max(2, min(4096, most)))
        return dict(op=op, layers=layers, pages=pages, pairs=rng.randint(1, pages // 2), heads=heads, dim=dim, page=page,
                    cache=cache, order=order)
    dim = rng.choice([64, 128, 256, 32 * rng.randint(1, 8)] if cache == "e4m3" else [64, 80, 128, 256, 8 * rng.randint(1, 32)])
    heads, q_heads = _heads(rng)
    seqs = _log(rng, 1, 128)
    length = _log(rng, 1, max(1, min(131072, (1 << 28) // (seqs * heads * dim))))
    return dict(op=op, seqs=seqs, q_heads=q_heads, heads=heads, dim=dim, page=page, length=length, ragged=rng.random() < 0.6,
                starts=rng.random() < 0.25, window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]),
                softcap=rng.choice([0.0, 0.0, 0.0, 20.0, 50.0]), type=kind, cache=cache, order=order)


# ---- inputs -----------------------------------------------------------------------------------

def _frequencies(case):
    """(angle per position of each pair, float64 array; factor on cos and sin)."""
    rot, base = case["rot"], 10000.0
    par = SCALINGS[case["scaling"]]
    i = np.arange(rot // 2, dtype=np.float64)
    if case["scaling"] == "ntk" and rot > 2:
        base *= par[0] ** (rot / (rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        f = f / par[0]
    if case["scaling"] == "bands":  # long waves are stretched, short ones kept, those between blended
        turns = par[1] * f / (2 * np.pi)
        keep = np.clip((turns - par[2]) / (par[3] - par[2]), 0.0, 1.0)
        f = (1 - keep) * f / par[0] + keep * f
    if case["scaling"] == "yarn":  # as above by pair index, and the logits' temperature
        at = [rot * math.log(par[1] / (t * 2 * math.pi)) / (2 * math.log(base)) for t in par[2:]]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return f / par[0] * ramp + f * (1 - ramp), 0.1 * math.log(par[0]) + 1.0
    return f, 1.0


def _shape(case, pages):
    inner = (case["heads"], case["page"]) if case["order"] == "heads" else (case["page"], case["heads"])
    return (pages, *inner, case["dim"])


def _plane(case, pages, g):
    """One plane (keys or values) of a cache in use: {"data"} or {"data": codes, "scale": E8M0}."""
    shape = _shape(case, pages)
    if case["cache"] != "e4m3":
        return {"data": torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[case["cache"]])}
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    scale = torch.empty((*shape[:3], shape[3] // 32), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
    for at in range(0, pages, step):
        x = torch.randn((min(step, pages - at), *shape[1:]), generator=g, device="cuda")
        codes[at:at + step], scale[at:at + step] = _quantise(x)
    return {"data": codes, "scale": scale}


def _quantise(x):
    """fp32 [..., dim] -> E4M3 codes and E8M0 scales per 32, both as bytes."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    fine = torch.isfinite(b).all(-1)
    e = torch.frexp(torch.where(fine, amax, 1.0)).exponent - 1 - 8 + 127
    e = torch.where(amax > 0, e.clamp(0, 254), 0)
    y = (b * torch.exp2((127 - e).to(torch.float32))[..., None]).clamp(-448.0, 448.0)
    codes = torch.where(fine[..., None], y, 0.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.reshape(x.shape), torch.where(fine, e, 255).to(torch.uint8)


def _held(plane):
    """A plane as the values that it holds: codes as E4M3 and scales as E8M0 numbers."""
    if "scale" not in plane:
        return [plane["data"]]
    return [plane["data"].view(torch.float8_e4m3fn), plane["scale"].view(torch.float8_e8m0fnu)]


def _table(case, lengths, pages, g):
    """Page tables of sequences of these lengths, their pages scattered over a cache of `pages` pages, -1 where none is."""
    page = case["page"]
    need = [-(-n // page) for n in lengths]
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(lengths), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    r = np.random.Generator(np.random.PCG64(int(seed)))
    s = {"case": case, "handles": None}
    if "rot" in case:
        f, s["factor"] = _frequencies(case)
        s["freq"] = torch.from_numpy(f).cuda()
    if case["op"] == "rotary":
        t, h, d, kind = case["tokens"], case["heads"], case["dim"], DTYPES[case["type"]]
        # the heads are a slice of a wider projection: the row's stride is not heads * dim
        s["x"] = torch.randn((t, h + 2, d), generator=g, device="cuda", dtype=kind)[:, :h]
        first = int(r.integers(0, max(1, case["far"] - t + 1)))
        s["positions"] = (torch.arange(t, dtype=torch.int32) + first).cuda()
        s["out"] = torch.empty((t, h, d), device="cuda", dtype=kind)
    elif case["op"] == "append":
        t, n, kind = case["tokens"], case["seqs"], DTYPES[case["type"]]
        # tokens per sequence: nearly equal for decode (one each), uneven for prompts
        cuts = np.sort(r.choice(np.arange(1, t), n - 1, replace=False)) if n > 1 else np.zeros(0, np.int64)
        counts = np.diff(np.concatenate([[0], cuts, [t]]))
        most = min(case["far"], max(1, (1 << 17) // n))
        first = r.integers(0, most, size=n)
        lengths = [int(a + c) for a, c in zip(first, counts)]
        page = case["page"]
        pages = n * -(-most // page) + t // page + n + 1  # enough for every draw of `first`
        s["table"] = _table(case, lengths, pages, g)
        s["seq"] = torch.from_numpy(np.repeat(np.arange(n), counts).astype(np.int32)).cuda()
        s["positions"] = torch.from_numpy(np.concatenate([np.arange(a, a + c) for a, c in zip(first, counts)]).astype(np.int32)).cuda()
        s["k_cache"], s["v_cache"] = _plane(case, pages, g), _plane(case, pages, g)
        hq, hk, d = case["q_heads"], case["heads"], case["dim"]
        qkv = torch.randn((t, hq + 2 * hk, d), generator=g, device="cuda", dtype=kind)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q_out"] = torch.empty((t, hq, d), device="cuda", dtype=kind)
        s["held"] = [_held(s["k_cache"]), _held(s["v_cache"])]
    elif case["op"] == "attention":
        n, most = case["seqs"], case["length"]
        lengths = np.full(n, most)
        if case["ragged"]:
            lengths = np.maximum(1, np.exp(r.uniform(math.log(max(1, most / 64)), math.log(most + 0.5), n)).astype(np.int64))
            lengths[int(r.integers(n))] = most
            if n > 4:
                lengths[int(r.integers(n))] = 0  # a slot of the batch that no request holds
        s["lengths"] = torch.from_numpy(lengths.astype(np.int32)).cuda()
        pages = int((-(-lengths // case["page"])).sum()) + 3
        s["table"] = _table(case, [int(x) for x in lengths], pages, g)
        s["starts"] = None
        if case["starts"]:  # padding on the left, which leaves one row nothing
            s["starts"] = torch.from_numpy(np.where((np.arange(n) == n - 1) & (n > 1), lengths, lengths // 3 * r.random(n)).astype(np.int32)).cuda()
        s["k_cache"], s["v_cache"] = _plane(case, pages, g), _plane(case, pages, g)
        hq, d, kind = case["q_heads"], case["dim"], DTYPES[case["type"]]
        s["q"] = torch.randn((n, hq, d), generator=g, device="cuda", dtype=kind)
        s["out"] = torch.empty((n, hq, d), device="cuda", dtype=kind)
        s["lse"] = torch.empty((n, hq), device="cuda", dtype=torch.float32)
        s["scale"] = d ** -0.5
    else:
        s["layers"] = [(_plane(case, case["pages"], g), _plane(case, case["pages"], g)) for _ in range(case["layers"])]
        order = torch.randperm(case["pages"], generator=g, device="cuda")[:2 * case["pairs"]]
        s["pairs"] = order.to(torch.int32).reshape(2, -1).t().contiguous()
        # what a copy hands back: at most eight of the layers, the first and the last among them
        last = case["layers"] - 1
        s["held"] = [_held(p) for i in sorted({round(j * last / 7) for j in range(8)}) for p in s["layers"][i]]
    return s


# ---- the plain forms --------------------------------------------------------------------------

def _rotated(s, x, inverse=False):
    """x [tokens, heads, dim] rotated by its tokens' positions, in fp32."""
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["factor"]).float()[:, None] for f in (torch.cos, torch.sin))
    if inverse:
        sin = -sin
    y, rot = x.float(), c["rot"]
    a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if c["layout"] == "half" else (y[..., 0:rot:2], y[..., 1:rot:2])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([u, v], -1) if c["layout"] == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _write(case, plane, page, slot, x):
    at = (page, slice(None), slot) if case["order"] == "heads" else (page, slot)
    if case["cache"] == "e4m3":
        plane["data"][at], plane["scale"][at] = _quantise(x.float())
    else:
        plane["data"][at] = x


def _read(case, plane, table):
    """The cache's values behind a table, [seqs, heads, positions, dim] in fp32."""
    pages = table.long().clamp(min=0)
    x = plane["data"][pages]
    if case["cache"] == "e4m3":
        scale = torch.exp2(plane["scale"][pages].float() - 127.0)
        x = x.view(torch.float8_e4m3fn).float()
        x = (x.reshape(*x.shape[:-1], -1, 32) * scale[..., None]).reshape(x.shape)
    x = x.float()
    if case["order"] == "heads":
        x = x.transpose(2, 3)
    return x.reshape(x.shape[0], -1, *x.shape[3:]).transpose(1, 2)


def _bounds(s):
    """First and last + 1 attended position of each sequence."""
    n = s["lengths"].long()
    first = torch.zeros_like(n) if s["starts"] is None else s["starts"].long()
    return torch.maximum(first, n - s["case"]["window"]) if s["case"]["window"] else first, n


def _attention(s):
    c = s["case"]
    n, hq, d = s["q"].shape
    k = _read(c, s["k_cache"], s["table"])
    q = s["q"].float().reshape(n, c["heads"], -1, d) * s["scale"]
    score = torch.matmul(q, k.transpose(2, 3).contiguous())
    del k
    if c["softcap"]:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    lo, hi = _bounds(s)
    at = torch.arange(score.shape[-1], device="cuda")
    seen = (at >= lo[:, None]) & (at < hi[:, None])
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, None, :, None], _read(c, s["v_cache"], s["table"]), 0.0)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return out.reshape(n, hq, d).to(s["q"].dtype), (top + torch.log(total)).reshape(n, hq)


def _plain(s):
    c = s["case"]
    if c["op"] == "rotary":
        return _rotated(s, s["x"], c["inverse"]).to(s["x"].dtype)
    if c["op"] == "append":
        page = s["table"][s["seq"].long(), (s["positions"] // c["page"]).long()].long()
        slot = (s["positions"] % c["page"]).long()
        _write(c, s["k_cache"], page, slot, _rotated(s, s["k"]).to(s["k"].dtype))
        _write(c, s["v_cache"], page, slot, s["v"])
        return _rotated(s, s["q"]).to(s["q"].dtype), *s["held"]
    if c["op"] == "attention":
        return _attention(s)
    src, dst = s["pairs"].long().unbind(1)
    for layer in s["layers"]:
        for plane in layer:
            for t in plane.values():
                t[dst] = t[src]
    return s["held"]


# ---- the package's operators ------------------------------------------------------------------

def _handles(s):
    """What a serving program keeps beside its tensors: the descriptors and a workspace."""
    from block_scaled_quantized_amd import api
    c = s["case"]
    fmt = {"fp16": api.MX_F16, "bf16": api.MX_BF16, "fp32": api.MX_F32, "e4m3": api.MX_E4M3}
    h = {"api": api, "type": fmt[c["type"]] if "type" in c else None}
    if "rot" in c:
        h["rope"] = api.Rope(c["rot"], s["freq"], api.MXROPE_HALF if c["layout"] == "half" else api.MXROPE_PAIRS, s["factor"])
    if "cache" in c:
        order = api.MXKV_HEADS_FIRST if c["order"] == "heads" else api.MXKV_SLOTS_FIRST
        both = s["layers"] if c["op"] == "copy" else [(s["k_cache"], s["v_cache"])]
        h["caches"] = [api.KVCache(fmt[c["cache"]], k["data"], v["data"], k.get("scale"), v.get("scale"), order=order) for k, v in both]
        if c["op"] == "copy":
            h["caches"] = api.kv_layers(h["caches"])
    if c["op"] == "attention":
        need = api.mxattn_decode_workspace_size(h["caches"][0], c["seqs"], c["q_heads"], c["length"])
        h["workspace"] = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")
    return h


def _own(s):
    c = s["case"]
    h = s["handles"] = s["handles"] or _handles(s)
    api = h["api"]
    if c["op"] == "rotary":
        api.mxrope_run(h["type"], h["rope"], s["x"], s["out"], s["positions"], inverse=c["inverse"])
        return s["out"]
    if c["op"] == "append":
        api.mxkv_append_run(h["caches"][0], h["type"], s["k"], s["v"], s["positions"], s["table"], seq=s["seq"], rope=h["rope"],
                            q=s["q"], q_out=s["q_out"])
        return s["q_out"], *s["held"]
    if c["op"] == "attention":
        api.mxattn_decode_run(h["caches"][0], h["type"], s["q"], s["out"], s["table"], s["lengths"], c["length"], s["scale"],
                              lse=s["lse"], starts=s["starts"], window=c["window"], softcap=c["softcap"], workspace=h["workspace"])
        return s["out"], s["lse"]
    api.mxkv_copy_run(h["caches"], s["pairs"])
    return s["held"]


def run(s):
    return _own(s) if own else _plain(s)


# ---- costs and the definition in 64 bits ------------------------------------------------------

def work(case):
    size = {"fp16": 2.0, "bf16": 2.0, "fp32": 4.0, "e4m3": 1 + 1 / 32}
    d = case["dim"]
    if case["op"] == "rotary":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * d * size[case["type"]] + 4 * case["tokens"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    if case["op"] == "append":
        t, hq, hk = case["tokens"], case["q_heads"], case["heads"]
        return {"bytes": t * d * (2 * (hq + hk) * size[case["type"]] + 2 * hk * size[case["cache"]]) + 12 * t,
                "flops": 3 * t * (hq + hk) * case["rot"]}
    if case["op"] == "copy":
        return {"bytes": 4 * case["layers"] * case["pairs"] * case["heads"] * case["page"] * d * size[case["cache"]], "flops": 0}
    n, most = case["seqs"], case["length"]
    keys = n * most
    if case["ragged"]:  # the mean of a log-uniform length
        lo = max(1.0, most / 64)
        keys = most + (n - 1) * ((most - lo) / math.log(most / lo) if most > lo else lo)
    if case["window"]:
        keys = min(keys, n * min(case["window"], most))
    return {"bytes": 2 * keys * case["heads"] * d * size[case["cache"]] + 2 * n * case["q_heads"] * d * size[case["type"]],
            "flops": 4 * keys * case["q_heads"] * d}


def exact(case, seed):
    if case["op"] == "copy":
        return None
    s = prepare(case, seed)

    def turn(x, sign=1.0):
        z = x.double()
        half = case["rot"] // 2
        one = torch.arange(half, device="cuda") * (1 if case["layout"] == "half" else 2)
        two = one + (half if case["layout"] == "half" else 1)
        w = s["positions"].double().unsqueeze(1) * s["freq"].unsqueeze(0) * sign
        by = torch.polar(torch.full_like(w, s["factor"]), w).unsqueeze(1)
        both = torch.complex(z[..., one], z[..., two]) * by
        z = z.clone()
        z[..., one], z[..., two] = both.real, both.imag
        return z

    if case["op"] == "rotary":
        return turn(s["x"], -1.0 if case["inverse"] else 1.0)
    if case["op"] == "append":
        q, k = turn(s["q"]), turn(s["k"])
        if case["cache"] == "e4m3":
            return q, [None, None], [None, None]
        planes = []
        for name, new in (("k_cache", k), ("v_cache", s["v"].double())):
            z = s[name]["data"].double()
            rows = z if case["order"] == "slots" else z.transpose(1, 2)
            where = s["positions"].long()
            page = s["table"].long()[s["seq"].long(), torch.div(where, case["page"], rounding_mode="floor")]
            rows[page, where.remainder(case["page"])] = new
            planes.append([z])
        return q, *planes
    n, hq, d = s["q"].shape
    out = torch.zeros((n, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    share = hq // case["heads"]
    for b in range(n):
        hi = int(s["lengths"][b])
        lo = int(s["starts"][b]) if s["starts"] is not None else 0
        lo = max(lo, hi - case["window"]) if case["window"] else lo
        if lo >= hi:
            continue
        row = s["table"][b, :-(-hi // case["page"])].long()
        kv = []
        for name in ("k_cache", "v_cache"):
            x = s[name]["data"][row]
            x = (x.view(torch.float8_e4m3fn).double() if case["cache"] == "e4m3" else x.double())
            if case["cache"] == "e4m3":
                x = x * torch.pow(2.0, s[name]["scale"][row].double() - 127).repeat_interleave(32, -1)
            x = x.permute(1, 0, 2, 3) if case["order"] == "heads" else x.permute(2, 0, 1, 3)
            kv.append(x.reshape(case["heads"], -1, d)[:, lo:hi])
        for h in range(case["heads"]):
            score = s["q"][b, h * share:(h + 1) * share].double() @ kv[0][h].t() * s["scale"]
            if case["softcap"]:
                score = case["softcap"] * torch.tanh(score / case["softcap"])
            lse[b, h * share:(h + 1) * share] = torch.logsumexp(score, -1)
            out[b, h * share:(h + 1) * share] = torch.softmax(score, -1) @ kv[1][h]
    return out, lse
