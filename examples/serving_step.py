"""A decoder's attention layer that serves a batch with 8-bit weights and activations, on cuda:0.

    python examples/serving_step.py [--cache e4m3|fp16] [--steps N] [--graph]

The layer: h = x + residual; qkv = norm(h) Wqkv in 8-bit integers; keys and values rotated and appended; x' = attention(q) Wo,
its operand quantised by rows; h is the next step's residual and x' its x. Rows 0 to 3 share a prompt, whose pages row 0 owns, rows 4 and 5 have
their own; every step gives each row that lives one token, and the pages for it are taken from a stack on the device, without the
host reading anything back, so that a step can be one captured graph (--graph). Half way row 4 ends and gives its pages
back. Every step's output is compared with the same layer in fp32 on contiguous keys and values; the largest difference is
printed.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_scaled_quantized_amd import api  # noqa: E402

HIDDEN, Q_HEADS, HEADS, DIM, PAGE, PAGES, SEQS, COLS = 512, 8, 2, 64, 16, 96, 6, 4096
WIDTH = (Q_HEADS + 2 * HEADS) * DIM
PROMPT, SHARING, OTHERS = 192, 4, (40, 75)  # tokens of the shared prompt, the rows that have it, the other rows' prompts


def empty(*shape, dtype=torch.float16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def ints(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Weights:
    """An 8-bit weight matrix [N][K] with a scale per output channel, and the values that it stands for."""

    def __init__(self, K, N, seed):
        w = (torch.randn(N, K, generator=torch.Generator().manual_seed(seed)) / K ** 0.5).half().cuda()
        self.K, self.N = K, N
        self.codes, self.scales = empty(N, K, dtype=torch.int8), empty(N, dtype=torch.float32)
        api.mxquant_rows_run(api.MX_F16, w, self.codes, self.scales, api.MX_INT8)
        self.values = (self.codes.float() * self.scales[:, None]).T.contiguous()

    def times(self, codes, scales, workspace):
        y = empty(codes.shape[0], self.N)
        api.mxgemm_i8_run(codes, scales, self.codes, self.scales, y, api.MX_F16, workspace=workspace)
        return y


class Step:
    """What mxkv_step_run writes for up to `most` new tokens."""

    def __init__(self, most):
        self.offsets, self.status = empty(SEQS + 1, dtype=torch.int32), ints(0)
        self.seq, self.positions, self.slots = (empty(most, dtype=torch.int32) for _ in range(3))


class Layer:
    """Weights, the cache with its pages' tables, and the buffers that a serving program keeps."""

    def __init__(self, kind):
        self.qkv, self.out = Weights(HIDDEN, WIDTH, 1), Weights(Q_HEADS * DIM, HIDDEN, 2)
        self.gain = (1 + torch.randn(HIDDEN, generator=torch.Generator().manual_seed(3)) / 8).half().cuda()
        freq, factor = api.mxrope_freqs_host(DIM, 10000.0)
        self.rope = api.Rope(DIM, torch.tensor(freq, dtype=torch.float64, device="cuda"), api.MXROPE_HALF, factor)
        shape = (PAGES, HEADS, PAGE, DIM)
        if kind == "e4m3":
            planes = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
            scales = [torch.zeros(*shape[:3], DIM // 32, dtype=torch.uint8, device="cuda") for _ in range(2)]
            self.cache = api.KVCache(api.MX_E4M3, *planes, *scales)
        else:
            self.cache = api.KVCache(api.MX_F16, *(torch.zeros(shape, dtype=torch.float16, device="cuda") for _ in range(2)))
        self.table = torch.full((SEQS, COLS), -1, dtype=torch.int32, device="cuda")
        self.lengths, self.kept = ints(*[0] * SEQS), ints(*[0] * SEQS)
        self.free, self.n_free = torch.arange(PAGES, dtype=torch.int32, device="cuda"), ints(PAGES)
        self.first, self.shared = ints(0, SHARING), ints(PROMPT)
        tokens = PROMPT + sum(OTHERS)
        need = [api.mxgemm_i8_workspace_size(m, w.N, w.K) for m in (tokens, SEQS) for w in (self.qkv, self.out)]
        need.append(api.mxattn_prefix_workspace_size(self.cache, SEQS, Q_HEADS, 1, COLS * PAGE, COLS * PAGE))
        # of each kind its own: products and attention keep different counters
        self.sums = torch.zeros(max(16, *need[:-1]), dtype=torch.uint8, device="cuda")
        self.splits = torch.zeros(max(16, need[-1]), dtype=torch.uint8, device="cuda")
        self.one, self.live = Step(SEQS), ints(*[1] * SEQS)

    def plan(self, step, wants):
        api.mxkv_step_run(PAGE, self.table, self.lengths, wants, self.free, self.n_free, step.offsets, step.seq, step.positions, step.slots,
                          step.status, kept=self.kept)

    def project(self, step, x, residual=None, decode=False):
        """Append the tokens of `step`, rows of x; their turned queries and the next residual."""
        codes, scales = empty(x.shape[0], HIDDEN, dtype=torch.int8), empty(x.shape[0], dtype=torch.float32)
        total = None if residual is None else torch.empty_like(x)
        api.mxnorm_run(api.MX_F16, x, codes, scales, api.MX_INT8, weight=self.gain, eps=1e-6, residual=residual, total=total)
        y = self.qkv.times(codes, scales, self.sums).view(x.shape[0], -1, DIM)
        q, k, v = y[:, :Q_HEADS], y[:, Q_HEADS:Q_HEADS + HEADS], y[:, Q_HEADS + HEADS:]
        turned = empty(*q.shape) if decode else None
        api.mxkv_append_run(self.cache, api.MX_F16, k, v, step.positions, self.table, seq=step.seq, rope=self.rope, q=q if decode else None, q_out=turned)
        return turned, total

    def prompts(self, shared, others):
        """The shared prompt goes to row 0, the others to rows SHARING on; rows 1 to SHARING - 1 then name row 0's pages."""
        x = torch.cat([shared, *others])
        step = Step(x.shape[0])
        self.plan(step, ints(PROMPT, *[0] * (SHARING - 1), *OTHERS))
        self.project(step, x)
        pages = PROMPT // PAGE
        self.table[1:SHARING, :pages] = self.table[0, :pages]
        self.lengths[1:SHARING] = PROMPT
        self.kept[:SHARING] = pages  # nobody gives them back while the others read them

    def step(self, x, residual):
        """One token of every row that lives; rows that do not end, and keep zeros. x, residual: [SEQS][HIDDEN]."""
        self.plan(self.one, torch.where(self.live > 0, self.lengths + 1, 0).int())
        row = self.one.seq.clamp(min=0).long()  # tokens are of the rows that grow, in order
        q, total = self.project(self.one, x[row], residual[row], True)
        token = self.one.offsets[:-1].clamp(max=SEQS - 1).long()
        o = empty(SEQS, Q_HEADS, DIM)
        api.mxattn_prefix_run(self.cache, api.MX_F16, q[token], o, self.table, self.lengths, COLS * PAGE, self.first, self.shared, COLS * PAGE,
                              DIM ** -0.5, workspace=self.splits)
        codes, scales = empty(SEQS, Q_HEADS * DIM, dtype=torch.int8), empty(SEQS, dtype=torch.float32)
        api.mxquant_rows_run(api.MX_F16, o.view(SEQS, -1), codes, scales, api.MX_INT8)
        return self.out.times(codes, scales, self.sums), total[token]


class Captured:
    """A layer's step as one graph on buffers of its own."""

    def __init__(self, layer):
        self.x, self.residual = (torch.zeros(SEQS, HIDDEN, dtype=torch.float16, device="cuda") for _ in range(2))
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = layer.step(self.x, self.residual)

    def __call__(self, x, residual):
        self.x.copy_(x)
        self.residual.copy_(residual)
        self.graph.replay()
        return tuple(t.clone() for t in self.out)


class Plain:
    """The same layer in fp32 torch operations with unquantised activations, each row's keys and values in one tensor."""

    def __init__(self, layer):
        self.wqkv, self.wo, self.gain = layer.qkv.values, layer.out.values, layer.gain.float()
        self.freq, self.kv = layer.rope.freq, [torch.zeros(2, 0, HEADS, DIM, device="cuda") for _ in range(SEQS)]

    def turn(self, x, pos):
        w = pos.double()[:, None] * self.freq
        cos, sin = w.cos().float()[:, None], w.sin().float()[:, None]
        a, b = x[..., :DIM // 2], x[..., DIM // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    def append(self, seq, h):
        h = h.float()
        y = (h * (h.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt() * self.gain) @ self.wqkv
        y = y.view(h.shape[0], -1, DIM)
        had = self.kv[seq].shape[1]
        pos = torch.arange(had, had + h.shape[0], device="cuda")
        self.kv[seq] = torch.cat([self.kv[seq], torch.stack([self.turn(y[:, Q_HEADS:Q_HEADS + HEADS], pos), y[:, Q_HEADS + HEADS:]])], 1)
        return self.turn(y[:, :Q_HEADS], pos)

    def step(self, seq, h):
        q = self.append(seq, h[None])[0].view(HEADS, -1, DIM)
        k, v = self.kv[seq].transpose(1, 2)
        p = torch.softmax(torch.matmul(q, k.transpose(1, 2).contiguous()) * DIM ** -0.5, -1)
        return torch.matmul(p, v).reshape(-1) @ self.wo


def main(kind="e4m3", steps=40, graph=False):
    """The largest difference between the layer's outputs and the plain form's, which are of size 1 or below, and the last outputs."""
    torch.manual_seed(0)
    layer = Layer(kind)
    plain = Plain(layer)
    prompts = [torch.randn(n, HIDDEN, device="cuda").half() for n in (PROMPT, *OTHERS)]
    layer.prompts(prompts[0], prompts[1:])
    for s in range(SEQS):
        plain.append(s, prompts[0 if s < SHARING else s - SHARING + 1])
    run = Captured(layer) if graph else layer.step
    x, residual = (torch.randn(SEQS, HIDDEN, device="cuda").half() for _ in range(2))
    live, worst = list(range(SEQS)), 0.0
    for i in range(steps):
        if i == steps // 2:
            live.remove(SHARING)
            layer.live[SHARING] = 0
        y, h = run(x, residual)
        assert layer.one.status.item() == 0
        for s in live:
            worst = max(worst, (y[s].float() - plain.step(s, (x[s].float() + residual[s].float()).half())).abs().max().item())
        x, residual = y, h
    used = sum(-(-n // PAGE) for n in layer.lengths.tolist()) - (SHARING - 1) * (PROMPT // PAGE)
    assert layer.n_free.item() == PAGES - used, "every page is in the table or on the stack"
    return worst, y


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--cache", choices=["e4m3", "fp16"], default="e4m3")
    p.add_argument("--steps", type=int, default=40)
    p.add_argument("--graph", action="store_true")
    a = p.parse_args()
    print(f"{a.steps} steps over a {a.cache} cache: largest difference from fp32 {main(a.cache, a.steps, a.graph)[0]:.5f}")
