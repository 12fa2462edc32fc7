"""Shared by the GPU tests of the decode step's cache: inputs, caches filled from numpy, page tables."""
import numpy as np
import torch

from gpu_common import require_gpu

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def fmt_of(api, kind):
    return {"f16": api.MX_F16, "bf16": api.MX_BF16, "f32": api.MX_F32, "e4m3": api.MX_E4M3}[kind]


def f64(t) -> np.ndarray:
    torch.cuda.synchronize()
    return t.detach().cpu().double().numpy()


def normal(shape, kind, seed, sigma=1.0):
    """A CUDA tensor of this type with N(0, sigma^2) values."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(TORCH[kind]).cuda()


class Cache:
    """A cache on the GPU, with what it holds as float64 in `k` and `v` ([pages][..][..][dim])."""

    def __init__(self, kind, order, pages, page, heads, dim, seed, fill=None, paired=False):
        self.api = api = require_gpu()
        self.kind, self.order, self.page, self.heads, self.dim = kind, order, page, heads, dim
        shape = (pages, heads, page, dim) if order == "heads" else (pages, page, heads, dim)
        self.planes, self.scales = [], []
        if kind == "e4m3":
            g = np.random.Generator(np.random.PCG64(seed))
            self.k, self.v = (np.zeros(shape) for _ in range(2))
            for want in (self.k, self.v):
                x = g.standard_normal(shape).astype(np.float32)
                if fill is not None:
                    x[:] = fill
                codes, scales = np.zeros(shape, np.uint8), np.zeros((*shape[:3], dim // 32), np.uint8)
                rows = x.size // dim
                api.mx_pack_host(api.MX_E4M3, x, rows, dim, codes, scales)
                back = np.zeros(shape, np.float32)
                api.mx_unpack_host(api.MX_E4M3, codes, scales, rows, dim, back)
                want[:] = back
                self.planes.append(torch.from_numpy(codes).cuda())
                self.scales.append(torch.from_numpy(scales).cuda())
        else:
            both = normal((pages, 2, *shape[1:]), kind, seed)
            if fill is not None:
                both.fill_(fill)
            self.planes = [both[:, 0], both[:, 1]] if paired else [both[:, 0].contiguous(), both[:, 1].contiguous()]
            self.k, self.v = (f64(t) for t in self.planes)
            self.scales = [None, None]
        self.c = api.KVCache(fmt_of(api, kind), *self.planes, *self.scales,
                             order=api.MXKV_HEADS_FIRST if order == "heads" else api.MXKV_SLOTS_FIRST)

    def rows(self, plane):
        """A plane (tensor or array) as [pages][page][heads][dim]."""
        return plane if self.order == "slots" else plane.swapaxes(1, 2)


def tables(lengths, page, pages, seed, cols=None):
    """int32 [seqs][cols] of distinct, scattered pages, -1 past each sequence's end."""
    need = [-(-n // page) for n in lengths]
    cols = cols or max(1, max(need))
    order = np.random.Generator(np.random.PCG64(seed)).permutation(pages)[:sum(need)]
    t, at = np.full((len(lengths), cols), -1, np.int32), 0
    for s, n in enumerate(need):
        t[s, :n] = order[at:at + n]
        at += n
    return t
