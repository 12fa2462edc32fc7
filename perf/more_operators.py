"""Cases and plain forms of a quantised serving step's operators: the RMS norm with the residual's addition and 8-bit outputs,
the product of 8-bit integers with a scale per token and channel, the step's page tables and slot maps, and the attention of a
batch whose rows share long beginnings.

`run` computes an operator in plain torch operations where `own` is false, and calls this package's entry points where it is
true. Page p of a sequence's table row holds its positions p * page .. p * page + page - 1, in [pages][heads][page][dim] ("heads")
or [pages][page][heads][dim] ("slots") order, as fp16 / bf16 values or as E4M3 codes with one E8M0 scale per 32 elements of dim.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # the residual stream of one decoded token, quantised for an MX product: launch latency
        dict(name="norm one token", op="norm", rows=1, dim=4096, type="fp16", residual=True, out="e4m3"),
        # a prompt's residual stream before an MX product
        dict(name="norm prompt", op="norm", rows=4096, dim=4096, type="bf16", residual=True, out="e4m3"),
        # a last norm in full precision over an odd width, unquantised
        dict(name="norm odd width", op="norm", rows=1777, dim=5003, type="fp32", residual=False, out="same"),
        # the widest projection of one decoded token: its weights are read once
        dict(name="product one token", op="product", M=1, N=14336, K=4096, out="fp16", bias=False, relu=False, pad=0),
        # a serving batch's projection, its activations normalised and quantised first
        dict(name="norm and product batch", op="linear", M=64, N=12288, K=4096, type="fp16", out="fp16", bias=False, residual=True),
        # a prompt's widest projection: the matrix cores
        dict(name="product prompt", op="product", M=2048, N=14336, K=4096, out="bf16", bias=False, relu=False, pad=0),
        # odd everything, with a bias and ReLU, rows longer than K
        dict(name="product odd", op="product", M=333, N=1003, K=2741, out="fp32", bias=True, relu=True, pad=32),
        # a decode step of a full batch: a token and now and then a page for each sequence
        dict(name="plan decode", op="plan", seqs=256, page=16, length=4096, tokens=256, back=False),
        # prompts that are admitted together, and given back
        dict(name="plan prompts", op="plan", seqs=37, page=64, length=8192, tokens=50000, back=True),
        # a few samples of one short prompt: latency
        dict(name="prefix short", op="prefix", seqs=4, groups=1, q_heads=32, heads=8, dim=128, page=16, prefix=1000, suffix=60,
             softcap=0.0, type="fp16", cache="fp16", order="heads"),
        # a batch behind one long system prompt
        dict(name="prefix batch", op="prefix", seqs=64, groups=1, q_heads=64, heads=8, dim=128, page=16, prefix=8192, suffix=512,
             softcap=0.0, type="bf16", cache="bf16", order="slots"),
        # several prompts with many samples each over a quantised cache, odd pages, capped scores
        dict(name="prefix groups e4m3", op="prefix", seqs=96, groups=5, q_heads=40, heads=8, dim=128, page=24, prefix=12000, suffix=1000,
             softcap=30.0, type="fp16", cache="e4m3", order="heads"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """Half of the sizes are multiples of 64, as models' are; the others are any."""
    n = _log(rng, lo, hi)
    return max(lo, min(hi, -(-n // 64) * 64)) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["norm", "product", "product", "linear", "plan", "prefix", "prefix"])
    kind = rng.choice(["fp16", "bf16"])
    if op == "norm":
        kind, out = rng.choice(["fp16", "bf16", "fp32"]), rng.choice(["e4m3", "e5m2", "same"])
        dim = _size(rng, 32, 16384)
        dim = dim if out == "same" else max(32, dim // 32 * 32)
        return dict(op=op, rows=_log(rng, 1, min(16384, (1 << 24) // dim)), dim=dim, type=kind, residual=rng.random() < 0.6, out=out)
    if op in ("product", "linear"):
        N, K = _size(rng, 16, 16384), _size(rng, 16, 16384)
        M = _log(rng, 1, min(8192, max(1, int(1.1e11) // (N * K))))
        case = dict(op=op, M=M, N=N, K=K, out=rng.choice(["fp16", "bf16"] if op == "linear" else ["fp16", "bf16", "fp32"]), bias=rng.random() < 0.3)
        return dict(case, type=kind, residual=rng.random() < 0.6) if op == "linear" else dict(case, relu=rng.random() < 0.3, pad=rng.choice([0, 0, 16, 64]))
    page = rng.choice([16, 32, 64, 128, 256, rng.randint(1, 100)])
    if op == "plan":
        seqs = _log(rng, 1, 2048)
        return dict(op=op, seqs=seqs, page=page, length=_log(rng, 1, 32768), tokens=_log(rng, 1, 65536), back=rng.random() < 0.4)
    cache = rng.choice([kind, "e4m3"])
    dim = rng.choice([64, 128, 256, 32 * rng.randint(1, 8)] if cache == "e4m3" else [64, 80, 128, 256, 8 * rng.randint(1, 32)])
    heads = rng.choice([1, 2, 3, 4, 8, 12, 16])
    q_heads = heads * rng.choice([1, 2, 4, 5, 7, 8, 16])
    seqs = _log(rng, 2, 256)
    groups = min(seqs // 2, _log(rng, 1, 16))
    prefix = _log(rng, 16, max(16, min(65536, (1 << 27) // (groups * heads * dim), (1 << 33) // (seqs * q_heads * dim))))
    return dict(op=op, seqs=seqs, groups=groups, q_heads=q_heads, heads=heads, dim=dim, page=page, prefix=prefix,
                suffix=_log(rng, 1, max(1, min(4096, (1 << 27) // (seqs * heads * dim)))), softcap=rng.choice([0.0, 0.0, 0.0, 20.0, 50.0]),
                type=kind, cache=cache, order=rng.choice(["heads", "slots"]))


# ---- inputs -----------------------------------------------------------------------------------

def _normal(shape, g, kind, sigma=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(DTYPES[kind])


def _stream_like(rows, dim, g, kind):
    """A residual stream: a few channels are far larger than the others."""
    x = torch.randn((rows, dim), generator=g, device="cuda")
    x[:, torch.randperm(dim, generator=g, device="cuda")[:max(1, dim // 512)]] *= 20.0
    return x.to(DTYPES[kind])


def _codes(shape, g):
    """8-bit codes of normal values, and the rows' scales: the largest of a row is at 127."""
    x = torch.randn(shape, generator=g, device="cuda")
    amax = x.abs().amax(-1, keepdim=True)
    return torch.round(x * (127.0 / amax)).to(torch.int8), (amax[:, 0] * (0.02 / 127.0)).contiguous()


def _padded(x, pad):
    """The same values in rows whose stride is a multiple of 16 bytes, `pad` more than it has to be."""
    rows = torch.zeros((x.shape[0], -(-x.shape[1] // 16) * 16 + pad), dtype=x.dtype, device="cuda")
    rows[:, :x.shape[1]] = x
    return rows[:, :x.shape[1]]


def _quantise(x, top=8, most=448.0, kind=torch.float8_e4m3fn):
    """fp32 [..., dim] -> 8-bit floating codes and E8M0 scales per 32, both as bytes."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    fine = torch.isfinite(b).all(-1)
    e = torch.frexp(torch.where(fine, amax, 1.0)).exponent - 1 - top + 127
    e = torch.where(amax > 0, e.clamp(0, 254), 0)
    y = (b * torch.exp2((127 - e).to(torch.float32))[..., None]).clamp(-most, most)
    codes = torch.where(fine[..., None], y, 0.0).to(kind).view(torch.uint8)
    return codes.reshape(x.shape), torch.where(fine, e, 255).to(torch.uint8)


E8 = {"e4m3": (8, 448.0, torch.float8_e4m3fn), "e5m2": (15, 57344.0, torch.float8_e5m2)}


def _plane(case, pages, g):
    """One plane (keys or values) of a cache in use: {"data"} or {"data": codes, "scale": E8M0}."""
    inner = (case["heads"], case["page"]) if case["order"] == "heads" else (case["page"], case["heads"])
    shape = (pages, *inner, case["dim"])
    if case["cache"] != "e4m3":
        return {"data": torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[case["cache"]])}
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    scale = torch.empty((*shape[:3], shape[3] // 32), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
    for at in range(0, pages, step):
        x = torch.randn((min(step, pages - at), *shape[1:]), generator=g, device="cuda")
        codes[at:at + step], scale[at:at + step] = _quantise(x)
    return {"data": codes, "scale": scale}


def _cuts(r, total, parts):
    """`parts` positive numbers of sum `total`."""
    at = np.sort(r.choice(np.arange(1, total), parts - 1, replace=False)) if parts > 1 else np.zeros(0, np.int64)
    return np.diff(np.concatenate([[0], at, [total]]))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    r = np.random.Generator(np.random.PCG64(int(seed)))
    s = {"case": case, "handles": None}
    op = case["op"]
    if op in ("norm", "linear"):
        rows, dim, kind = (case["rows"], case["dim"], case["type"]) if op == "norm" else (case["M"], case["K"], case["type"])
        # rows of a multiple of 16 bytes, as an allocation for such kernels has
        unit = 16 // DTYPES[kind].itemsize
        wide = -(-dim // unit) * unit
        s["x"] = _stream_like(rows, wide, g, kind)[:, :dim]
        s["residual"] = _stream_like(rows, wide, g, kind)[:, :dim] if case["residual"] else None
        s["total"] = torch.zeros((rows, wide), dtype=DTYPES[kind], device="cuda")[:, :dim] if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(DTYPES[kind])
    if op == "norm":
        if case["out"] == "same":
            s["out"], s["scales"] = torch.zeros((rows, wide), dtype=DTYPES[kind], device="cuda")[:, :dim], None
        else:
            s["out"] = torch.zeros((rows, dim), dtype=torch.uint8, device="cuda")
            s["scales"] = torch.zeros((rows, dim // 32), dtype=torch.uint8, device="cuda")
    if op in ("product", "linear"):
        M, N, K = case["M"], case["N"], case["K"]
        b, s["sb"] = _codes((N, K), g)
        s["b"] = _padded(b, case.get("pad", 0))
        if op == "product":
            a, s["sa"] = _codes((M, K), g)
            s["a"] = _padded(a, case["pad"])
        else:
            s["a"], s["sa"] = _padded(torch.zeros((M, K), dtype=torch.int8, device="cuda"), 0), torch.zeros(M, device="cuda")
        s["bias"] = _normal((N,), g, case["out"]) if case["bias"] else None
        s["c"] = torch.zeros((M, N), dtype=DTYPES[case["out"]], device="cuda")
    if op == "plan":
        n, page, most = case["seqs"], case["page"], case["length"]
        has = r.integers(0, most + 1, size=n)
        if n > 2:
            has[r.integers(n, size=n // 3)] = 0  # places of the batch that no request held yet
        count = np.zeros(n, np.int64)
        if case["tokens"] <= n:
            count[r.choice(n, case["tokens"], replace=False)] = 1
        else:
            live = r.choice(n, max(1, n * 3 // 4), replace=False)
            count[live] = _cuts(r, case["tokens"], len(live))
        need, after = -(-has // page), -(-(has + count) // page)
        # a table for the longest row that the sizes allow, and pages enough for all
        cols = -(-(most + case["tokens"]) // page)
        pages = n * -(-most // page) + case["tokens"] // page + n + 1
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        held = int(need.sum())
        table = torch.full((n, cols), -1, dtype=torch.int32)
        flat = order[:held].cpu()
        at = 0
        for b in range(n):
            table[b, :need[b]] = flat[at:at + int(need[b])]
            at += int(need[b])
        s["table"] = table.cuda()
        s["free"] = torch.cat([order[held:], torch.zeros(held, dtype=torch.int32, device="cuda")])
        s["n_free"] = torch.tensor([pages - held], dtype=torch.int32, device="cuda")
        s["has"] = torch.from_numpy(has.astype(np.int32)).cuda()
        s["wants"] = torch.from_numpy((has + count).astype(np.int32)).cuda()
        # a batch padded for a captured step: places behind the last token
        s["room"] = case["tokens"] + (-case["tokens"]) % 64
        s["lengths"], s["left"] = torch.zeros_like(s["has"]), torch.zeros_like(s["n_free"])
        s["offsets"] = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
        s["maps"] = [torch.zeros(s["room"], dtype=torch.int32, device="cuda") for _ in range(3)]
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["spare"] = [torch.zeros_like(t) for t in (s["offsets"], *s["maps"], s["status"])]
    if op == "prefix":
        n, groups, page = case["seqs"], case["groups"], case["page"]
        members = _cuts(r, n, groups)
        first = np.concatenate([[0], np.cumsum(members)])
        whole = case["prefix"] // page  # pages of the longest shared beginning
        own_pages = np.maximum(1, (whole * np.exp(r.uniform(-1.0, 0.0, groups))).astype(np.int64)) if whole else np.zeros(groups, np.int64)
        if whole:
            own_pages[int(r.integers(groups))] = whole
        shared = own_pages * page
        suffix = r.integers(1, case["suffix"] + 1, size=n)
        suffix[int(r.integers(n))] = case["suffix"]
        cols = whole + -(-case["suffix"] // page)
        pages = int(groups * whole + n * -(-case["suffix"] // page)) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu().numpy()
        table, lengths, at = np.full((n, cols), -1, np.int32), np.zeros(n, np.int64), 0
        for i in range(groups):
            common = order[at:at + own_pages[i]]
            at += int(own_pages[i])
            for b in range(first[i], first[i + 1]):
                rest = int(-(-suffix[b] // page))
                table[b, :own_pages[i]] = common
                table[b, own_pages[i]:own_pages[i] + rest] = order[at:at + rest]
                at += rest
                lengths[b] = shared[i] + suffix[b]
        if n > 4 and members.max() > 1:  # a place of the batch that no request holds
            lengths[first[int(members.argmax()) + 1] - 1] = 0
        s["table"], s["lengths"] = torch.from_numpy(table).cuda(), torch.from_numpy(lengths.astype(np.int32)).cuda()
        s["first"], s["shared"] = (torch.from_numpy(t.astype(np.int32)).cuda() for t in (first, shared))
        s["most"], s["longest"], s["members"] = int(whole * page), cols * page, int(members.max())
        s["k_cache"], s["v_cache"] = _plane(case, pages, g), _plane(case, pages, g)
        s["q"] = _normal((n, case["q_heads"], case["dim"]), g, case["type"])
        s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros(s["q"].shape[:2], device="cuda")
        s["scale"] = case["dim"] ** -0.5
    return s


# ---- the plain forms --------------------------------------------------------------------------

def _normed(s):
    """(x + residual in its type, the norm in fp32)."""
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    z = h.float()
    return h, z * torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS) * s["weight"].float()


def _product(a, sa, s):
    c = torch.matmul(a, s["b"].float().t()) * sa[:, None] * s["sb"]
    if s["bias"] is not None:
        c = c + s["bias"].float()
    return (torch.clamp(c, min=0.0) if s["case"].get("relu") else c).to(DTYPES[s["case"]["out"]])


def _planned(s, has, wants, table, free, n_free):
    """Table, lengths, free stack and count after the step, and its tokens' rows, positions and slots."""
    page, cols = s["case"]["page"], table.shape[1]
    a, b = ((t.long() + page - 1) // page for t in (has, wants))
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    at = torch.arange(cols, device="cuda")
    gives, takes = (at >= b[:, None]) & (at < a[:, None]), (at >= a[:, None]) & (at < b[:, None])
    n_give = gives.sum()
    rank = torch.cumsum(gives.flatten().long(), 0).view(gives.shape) - 1
    free = free.clone()
    place = torch.where(gives, n_free.long() + n_give - 1 - rank, free.numel())
    free = torch.cat([free, zero.int()]).scatter(0, place.flatten(), table.flatten())[:-1]
    rank = torch.cumsum(takes.flatten().long(), 0).view(takes.shape) - 1
    top = n_free.long() + n_give
    got = free[(top - 1 - rank).clamp(0, free.numel() - 1).flatten()].view(takes.shape)
    table = torch.where(takes, got, torch.where(gives, -1, table))
    offsets = torch.cat([zero, torch.cumsum((wants - has).clamp(min=0).long(), 0)])
    t = torch.arange(s["room"], device="cuda")
    row = torch.searchsorted(offsets, t, right=True) - 1
    live = t < offsets[-1]
    row = torch.where(live, row, 0)
    pos = has.long()[row] + t - offsets[row]
    slot = table[row, (pos // page).clamp(0, cols - 1)].long() * page + pos % page
    maps = [torch.where(live, v, -1).int() for v in (row, pos, slot)]
    return table, wants.clone(), free, (top - takes.sum()).int(), offsets.int(), maps


def _plan(s):
    table, lengths, free, left, offsets, maps = _planned(s, s["has"], s["wants"], s["table"], s["free"], s["n_free"])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if s["case"]["back"]:
        table, lengths, free, left, _, _ = _planned(s, lengths, s["has"], table, free, left)
    return table, lengths, left, free, offsets, maps, status


def _read(case, plane, table):
    """The cache's values behind a table, [rows, heads, positions, dim] in fp32."""
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


def _attend(c, q, k, v, seen):
    """Maximum, sum and unscaled output of q [rows][heads][m][dim] over the seen keys; seen: [rows][1][1][keys]."""
    score = torch.matmul(q, k.transpose(2, 3).contiguous())
    if c["softcap"]:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    return top, p.sum(-1, keepdim=True), torch.matmul(p, torch.where(seen.transpose(2, 3), v, 0.0))


def _prefix(s):
    c = s["case"]
    n, hq, d = s["q"].shape
    heads, share, page = c["heads"], hq // c["heads"], c["page"]
    first, shared, lengths = s["first"].long(), s["shared"].long(), s["lengths"].long()
    row = torch.arange(n, device="cuda")
    group = torch.searchsorted(first, row, right=True) - 1
    place = row - first[group]
    q = s["q"].float().reshape(n, heads, share, d) * s["scale"]
    # the shared positions: every group's rows together, in as many places as its largest has
    both = None
    if s["most"]:
        rows = torch.zeros((len(shared), s["members"], heads, share, d), device="cuda")
        rows[group, place] = q
        rows = rows.permute(0, 2, 1, 3, 4).reshape(len(shared), heads, -1, d)
        pages = s["table"][first[:-1]][:, :s["most"] // page]
        at = torch.arange(pages.shape[1] * page, device="cuda")
        seen = (at < shared[:, None])[:, None, None]
        both = _attend(c, rows, _read(c, s["k_cache"], pages), _read(c, s["v_cache"], pages), seen)
        both = [t.view(len(shared), heads, s["members"], share, -1).permute(0, 2, 1, 3, 4)[group, place] for t in both]
        empty = (lengths == 0)[:, None, None, None]
        both = [torch.where(empty, -math.inf, both[0]), torch.where(empty, 0.0, both[1]), torch.where(empty, 0.0, both[2])]
    # each row's own positions
    begin = shared[group] // page
    wide = -(-c["suffix"] // page)
    cols = (begin[:, None] + torch.arange(wide, device="cuda")).clamp(max=s["table"].shape[1] - 1)
    pages = torch.gather(s["table"], 1, cols)
    at = begin[:, None] * page + torch.arange(wide * page, device="cuda")
    seen = (at < lengths[:, None])[:, None, None]
    top, total, out = _attend(c, q, _read(c, s["k_cache"], pages), _read(c, s["v_cache"], pages), seen)
    if both is not None:
        m = torch.maximum(top, both[0])
        ref = torch.where(torch.isinf(m), 0.0, m)
        x, y = torch.exp(top - ref), torch.exp(both[0] - ref)
        top, total, out = m, total * x + both[1] * y, out * x + both[2] * y
    out = out / torch.where(total > 0, total, 1.0)
    return out.reshape(n, hq, d).to(s["q"].dtype), (top + torch.log(total)).reshape(n, hq)


def _plain(s):
    c = s["case"]
    if c["op"] == "product":
        return _product(s["a"].float(), s["sa"], s)
    if c["op"] == "plan":
        return _plan(s)
    if c["op"] == "prefix":
        return _prefix(s)
    h, y = _normed(s)
    if c["op"] == "linear":
        amax = y.abs().amax(-1, keepdim=True)
        q = torch.round(y * (127.0 / torch.where(amax > 0, amax, 1.0)))
        out = [_product(q, amax[:, 0] / 127.0, s)]
    elif c["out"] == "same":
        out = [y.to(s["x"].dtype)]
    else:
        codes, scale = _quantise(y, *E8[c["out"]])
        out = [codes.view(E8[c["out"]][2]), scale.view(torch.float8_e8m0fnu)]
    return out + ([h] if c["residual"] else [])


# ---- the package's operators ------------------------------------------------------------------

def _handles(s):
    """What a serving program keeps beside its tensors: the cache's descriptor and workspaces."""
    from block_scaled_quantized_amd import api
    c = s["case"]
    fmt = {"fp16": api.MX_F16, "bf16": api.MX_BF16, "fp32": api.MX_F32, "e4m3": api.MX_E4M3, "e5m2": api.MX_E5M2}
    fmt["same"] = fmt.get(c.get("type"))
    h = {"api": api, "fmt": fmt}
    if c["op"] in ("product", "linear"):
        need = api.mxgemm_i8_workspace_size(c["M"], c["N"], c["K"])
        h["workspace"] = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")
    if c["op"] == "prefix":
        order = api.MXKV_HEADS_FIRST if c["order"] == "heads" else api.MXKV_SLOTS_FIRST
        k, v = s["k_cache"], s["v_cache"]
        h["cache"] = api.KVCache(fmt[c["cache"]], k["data"], v["data"], k.get("scale"), v.get("scale"), order=order)
        need = api.mxattn_prefix_workspace_size(h["cache"], c["seqs"], c["q_heads"], c["groups"], s["longest"], max(1, s["most"]))
        h["workspace"] = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")
    return h


def _own(s):
    c = s["case"]
    h = s["handles"] = s["handles"] or _handles(s)
    api, fmt = h["api"], h["fmt"]
    if c["op"] == "plan":
        if not c["back"]:
            api.mxkv_step_run(c["page"], s["table"], s["has"], s["wants"], s["free"], s["n_free"], s["offsets"], *s["maps"], s["status"],
                              lengths_out=s["lengths"], n_free_out=s["left"])
        else:  # taken and given back: the table and the stack end as they began
            api.mxkv_step_run(c["page"], s["table"], s["has"], s["wants"], s["free"], s["n_free"], s["offsets"], *s["maps"], s["status"],
                              lengths_out=s["lengths"], n_free_out=s["left"])
            api.mxkv_step_run(c["page"], s["table"], s["lengths"], s["has"], s["free"], s["left"], *s["spare"])
        return s["table"], s["lengths"], s["left"], s["free"], s["offsets"], s["maps"], s["status"]
    if c["op"] == "prefix":
        api.mxattn_prefix_run(h["cache"], fmt[c["type"]], s["q"], s["out"], s["table"], s["lengths"], s["longest"], s["first"], s["shared"],
                              max(1, s["most"]), s["scale"], lse=s["lse"], softcap=c["softcap"], workspace=h["workspace"])
        return s["out"], s["lse"]
    more = [s["total"]] if c.get("residual") else []
    if c["op"] == "norm":
        api.mxnorm_run(fmt[c["type"]], s["x"], s["out"], s["scales"], fmt[c["out"]], weight=s["weight"], eps=EPS, residual=s["residual"], total=s["total"])
        if c["out"] == "same":
            return [s["out"]] + more
        return [s["out"].view(E8[c["out"]][2]), s["scales"].view(torch.float8_e8m0fnu)] + more
    if c["op"] == "linear":
        api.mxnorm_run(fmt[c["type"]], s["x"], s["a"], s["sa"], api.MX_INT8, weight=s["weight"], eps=EPS, residual=s["residual"], total=s["total"])
    api.mxgemm_i8_run(s["a"], s["sa"], s["b"], s["sb"], s["c"], fmt[c["out"]], bias=s["bias"], flags=api.MXGEMM_RELU if c.get("relu") else 0,
                      workspace=h["workspace"])
    return [s["c"]] + more if c["op"] == "linear" else s["c"]


def run(s):
    return _own(s) if own else _plain(s)


# ---- costs and the definition in 64 bits ------------------------------------------------------

def work(case):
    size = {"fp16": 2.0, "bf16": 2.0, "fp32": 4.0, "e4m3": 1 + 1 / 32, "e5m2": 1 + 1 / 32}
    op = case["op"]
    if op == "norm":
        n, x = case["rows"] * case["dim"], size[case["type"]]
        return {"bytes": n * (x * (3 if case["residual"] else 1) + size.get(case["out"], x)) + case["dim"] * x, "flops": 5 * n}
    if op in ("product", "linear"):
        M, N, K = case["M"], case["N"], case["K"]
        fixed = N * K + 4 * N + M * N * size[case["out"]] + (N * size[case["out"]] if case["bias"] else 0)
        if op == "product":
            return {"bytes": fixed + M * K + 4 * M, "flops": 2 * M * N * K}
        return {"bytes": fixed + M * K * size[case["type"]] * (3 if case["residual"] else 1) + K * size[case["type"]], "flops": 2 * M * N * K}
    if op == "plan":
        moved = case["tokens"] / case["page"] + min(case["tokens"], case["seqs"]) / 2  # pages
        once = 4 * (4 * case["seqs"] + 3 * case["tokens"] + 2 * moved)
        return {"bytes": once + (4 * (3 * case["seqs"] + 3 * moved) if case["back"] else 0), "flops": 0}
    n, d = case["seqs"], case["dim"]
    shared = case["prefix"] * (1 if case["groups"] == 1 else 0.7)  # the mean over groups
    keys = case["groups"] * shared + n * case["suffix"] / 2
    return {"bytes": 2 * keys * case["heads"] * d * size[case["cache"]] + 2 * n * case["q_heads"] * d * size[case["type"]],
            "flops": 4 * n * (shared + case["suffix"] / 2) * case["q_heads"] * d}


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)

    def times(a, sa):
        c = torch.einsum("mk,nk->mn", a.double(), s["b"].double())
        c *= torch.outer(sa.double(), s["sb"].double())
        if case["bias"]:
            c += s["bias"].double().unsqueeze(0)
        return c.clamp_(min=0) if case.get("relu") else c

    if case["op"] == "product":
        return times(s["a"], s["sa"])
    if case["op"] in ("norm", "linear"):
        h = s["x"].double()
        if case["residual"]:
            h = (h + s["residual"].double()).to(s["x"].dtype).double()
        y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / h.shape[1] + EPS) * s["weight"].double().unsqueeze(0)
        more = [h] if case["residual"] else []
        if case["op"] == "linear":
            step = y.abs().max(1).values / 127
            return [times(torch.round(y / step.unsqueeze(1)), step)] + more
        if case["out"] == "same":
            return [y] + more
        blocks = y.unflatten(1, (-1, 32))
        step = torch.exp2(torch.floor(torch.log2(blocks.abs().max(2).values)) - {"e4m3": 8, "e5m2": 15}[case["out"]])
        codes = (blocks / step.unsqueeze(2)).flatten(1)
        most = {"e4m3": 448.0, "e5m2": 57344.0}[case["out"]]
        return [codes.clamp(-most, most), step] + more
    n, hq, d = s["q"].shape
    share = hq // case["heads"]
    out = torch.zeros((n, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")

    def held(name, pages):
        x = s[name]["data"][pages]
        x = x.view(torch.float8_e4m3fn).double() if case["cache"] == "e4m3" else x.double()
        if case["cache"] == "e4m3":
            x = x * torch.pow(2.0, s[name]["scale"][pages].double() - 127).repeat_interleave(32, -1)
        x = x.permute(1, 0, 2, 3) if case["order"] == "heads" else x.permute(2, 0, 1, 3)
        return x.reshape(case["heads"], -1, d)

    # a row's whole length as its own attention: what is shared is in its table as well
    for b in range(n):
        length = int(s["lengths"][b])
        if length == 0:
            continue
        pages = s["table"][b, :-(-length // case["page"])].long()
        k, v = held("k_cache", pages)[:, :length], held("v_cache", pages)[:, :length]
        q = s["q"][b].double().view(case["heads"], share, d)
        score = torch.bmm(q, k.transpose(1, 2).contiguous()) * s["scale"]
        if case["softcap"]:
            score = case["softcap"] * torch.tanh(score / case["softcap"])
        lse[b] = torch.logsumexp(score, -1).flatten()
        out[b] = torch.bmm(torch.softmax(score, -1), v).flatten(0, 1)
    return out, lse
