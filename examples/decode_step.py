"""An attention layer that decodes with int8 weights over a paged E4M3 cache, on cuda:0.

    python examples/decode_step.py [--cache e4m3|fp16] [--steps N]

The layer: qkv = x Wqkv; keys and values rotated and appended; out = attention(q) Wo; the next step's x is the
normalised sum. Two prompts are appended in one call each, a third sequence forks from the first (its pages
are shared, and the last one copied when either grows), every step decodes one token of each, half way
the first prompt ends and the cache is compacted. Every step's output is compared with the same layer in fp32 on a
contiguous cache; the largest difference is printed.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_scaled_quantized_amd import api  # noqa: E402

HIDDEN, Q_HEADS, HEADS, DIM, PAGE, PAGES, SEQS, COLS = 512, 8, 2, 64, 16, 48, 3, 12
WIDTH = (Q_HEADS + 2 * HEADS) * DIM


class Weights:
    """An int8 weight matrix [K][N] with fp16 scales per 32 rows, and the values that it stands for."""

    def __init__(self, K, N, seed):
        w = torch.randn(K, N, generator=torch.Generator().manual_seed(seed)) / K ** 0.5
        self.K, self.N = K, N
        self.codes = torch.empty(K, N, dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(K // 32, N, dtype=torch.float16, device="cuda")
        api.mx_pack_run(api.MX_INT8, w.cuda(), K, N, self.codes, self.scales)
        self.values = self.codes.view(torch.int8).float() * self.scales.float().repeat_interleave(32, 0)

    def times(self, x):
        y = torch.empty(x.shape[0], self.N, dtype=torch.float16, device="cuda")
        api.mxmatvec_run(x.shape[0], self.N, self.K, x, self.codes, api.MX_INT8, self.scales, y)
        return y


class Layer:
    """Weights, one layer's cache with its page pool, and the buffers that a serving program keeps."""

    def __init__(self, kind):
        self.qkv, self.out = Weights(HIDDEN, WIDTH, 1), Weights(Q_HEADS * DIM, HIDDEN, 2)
        freq, factor = api.mxrope_freqs_host(DIM, 10000.0)
        self.rope = api.Rope(DIM, torch.tensor(freq, dtype=torch.float64, device="cuda"), api.MXROPE_HALF, factor)
        shape = (PAGES, HEADS, PAGE, DIM)
        if kind == "e4m3":
            planes = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
            scales = [torch.zeros(*shape[:3], DIM // 32, dtype=torch.uint8, device="cuda") for _ in range(2)]
            self.cache = api.KVCache(api.MX_E4M3, *planes, *scales)
        else:
            planes = [torch.zeros(shape, dtype=torch.float16, device="cuda") for _ in range(2)]
            self.cache = api.KVCache(api.MX_F16, *planes)
        self.pool = api.KVPool(PAGES, PAGE, SEQS, COLS)
        need = api.mxattn_decode_workspace_size(self.cache, SEQS, Q_HEADS, COLS * PAGE)
        self.workspace = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")

    def copy(self, pairs):
        if pairs:
            api.mxkv_copy_run([self.cache], torch.tensor(pairs, dtype=torch.int32, device="cuda"))

    def project(self, x, seq, first, decode):
        """Append the rows of x, tokens of sequence seq[i] at position first[i]; the turned queries."""
        y = self.qkv.times(x).view(x.shape[0], -1, DIM)
        q, k, v = y[:, :Q_HEADS], y[:, Q_HEADS:Q_HEADS + HEADS], y[:, Q_HEADS + HEADS:]
        table = torch.from_numpy(self.pool.table()).cuda()
        pos, rows = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in (first, seq))
        turned = torch.empty(q.shape, dtype=torch.float16, device="cuda") if decode else None
        api.mxkv_append_run(self.cache, api.MX_F16, k, v, pos, table, seq=rows, rope=self.rope, q=q if decode else None, q_out=turned)
        return turned, table

    def prompt(self, seq, x):
        self.copy(self.pool.resize(seq, x.shape[0]))
        self.project(x, [seq] * x.shape[0], list(range(x.shape[0])), False)

    def step(self, x, live):
        """One token of every sequence in `live` (x: [SEQS][HIDDEN]; other rows are ignored)."""
        at = [int(n) for n in self.pool.lengths()]
        for s in live:
            self.copy(self.pool.resize(s, at[s] + 1))
        q, table = self.project(x, list(range(SEQS)), [at[s] if s in live else -1 for s in range(SEQS)], True)
        lengths = torch.from_numpy(self.pool.lengths()).cuda()
        o = torch.empty(SEQS, Q_HEADS, DIM, dtype=torch.float16, device="cuda")
        api.mxattn_decode_run(self.cache, api.MX_F16, q, o, table, lengths, COLS * PAGE, DIM ** -0.5, workspace=self.workspace)
        return self.out.times(o.view(SEQS, -1))


class Plain:
    """The same layer in fp32 torch operations, each sequence's keys and values in one tensor."""

    def __init__(self, layer):
        self.wqkv, self.wo, self.kv = layer.qkv.values, layer.out.values, [None] * SEQS
        self.freq = layer.rope.freq

    def turn(self, x, pos):
        w = pos.double()[:, None] * self.freq
        cos, sin = w.cos().float()[:, None], w.sin().float()[:, None]
        a, b = x[..., :DIM // 2], x[..., DIM // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    def append(self, seq, x):
        y = (x.float() @ self.wqkv).view(x.shape[0], -1, DIM)
        had = 0 if self.kv[seq] is None else self.kv[seq].shape[1]
        pos = torch.arange(had, had + x.shape[0], device="cuda")
        kv = torch.stack([self.turn(y[:, Q_HEADS:Q_HEADS + HEADS], pos), y[:, Q_HEADS + HEADS:]])
        self.kv[seq] = kv if had == 0 else torch.cat([self.kv[seq], kv], 1)
        return self.turn(y[:, :Q_HEADS], pos)

    def step(self, seq, x):
        q = self.append(seq, x[None])[0].view(HEADS, -1, DIM)
        k, v = self.kv[seq].transpose(1, 2)
        p = torch.softmax(torch.matmul(q, k.transpose(1, 2).contiguous()) * DIM ** -0.5, -1)
        return torch.matmul(p, v).reshape(-1) @ self.wo


def main(kind="e4m3", steps=24):
    """The largest difference between the layer's outputs and the plain form's, which are of size 1 or below."""
    torch.manual_seed(0)
    layer = Layer(kind)
    plain = Plain(layer)
    for s, n in ((0, 37), (1, 70)):
        x = torch.randn(n, HIDDEN, device="cuda").half()
        layer.prompt(s, x)
        plain.append(s, x)
    layer.pool.fork(0, 2)
    plain.kv[2] = plain.kv[0].clone()
    live, worst = [0, 1, 2], 0.0
    x = torch.randn(SEQS, HIDDEN, device="cuda").half()
    for i in range(steps):
        if i == steps // 2:
            live = [1, 2]
            layer.pool.resize(0, 0)
            layer.copy(layer.pool.compact())
        y = layer.step(x, live)
        for s in live:
            worst = max(worst, (y[s].float() - plain.step(s, x[s])).abs().max().item())
        z = x.float() + y.float()
        x = (z / z.pow(2).mean(-1, keepdim=True).sqrt()).half()
    return worst


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--cache", choices=["e4m3", "fp16"], default="e4m3")
    p.add_argument("--steps", type=int, default=24)
    a = p.parse_args()
    print(f"{a.steps} steps over a {a.cache} cache: largest difference from fp32 {main(a.cache, a.steps):.5f}")
