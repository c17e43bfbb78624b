"""A small decoder on the library: Q8_0 projections, the paged key-value cache and its attention together.

    python examples/cached_decoder.py

Prompts of different lengths are prefilled in one packed call, one of them is forked into two branches, all
sequences decode token by token, a branch is released and the pool compacted on the way.  At the end the same
hidden states are computed without a cache, as whole prompts, and compared.  Weights are random.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import inputs
import q8_quantized_matmul_gb300 as q8

DIM, HEADS, KV, HEAD, MID, LAYERS, PAGE = 1024, 8, 2, 128, 2048, 2, 16
EPS, THETA, MAX_POS = 1e-6, 10000.0, 4096


class Decoder:
    def __init__(self, seed=0):
        def weight(rows, cols, s):   # Q8_0 rows, standard deviation about 1/32
            w = inputs.weights(rows, cols, seed=seed * 100 + s, d_lo=3e-4, d_hi=5.5e-4)
            return torch.from_numpy(w).cuda()
        self.layers = [dict(qkv=weight((HEADS + 2 * KV) * HEAD, DIM, 10 * i), out=weight(DIM, HEADS * HEAD, 10 * i + 1),
                            gate=weight(MID, DIM, 10 * i + 2), up=weight(MID, DIM, 10 * i + 3),
                            down=weight(DIM, MID, 10 * i + 4)) for i in range(LAYERS)]
        f = THETA ** (-torch.arange(HEAD // 2, dtype=torch.float64, device="cuda") / (HEAD // 2))
        a = torch.arange(MAX_POS, dtype=torch.float64, device="cuda")[:, None] * f
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float()

    def forward(self, x, positions, attend):
        """x fp32 [n, DIM]; attend(layer, q, k, v) takes the fp32 projections and gives Q8_0 blocks [n, ...]."""
        n = x.shape[0]
        for i, w in enumerate(self.layers):
            h = q8.rmsnorm_quantize(x, None, EPS)
            qkv = q8.matmul_q(w["qkv"], h, DIM, (HEADS + 2 * KV) * HEAD).view(n, -1, HEAD)
            o = attend(i, qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:])
            x = x + q8.matmul_q(w["out"], o.view(n, -1), HEADS * HEAD, DIM)
            h = q8.rmsnorm_quantize(x, None, EPS)
            gate, up = (q8.matmul_q(w[k], h, DIM, MID) for k in ("gate", "up"))
            mid = torch.empty_like(gate)
            assert q8.q8_swiglu(mid, gate, up, mid.numel(), 0.0) == q8.Q8_OK
            x = x + q8.matmul(w["down"], mid, DIM)
        return x


class Server:
    """Sequences in a paged cache: rows of a table, page counts, lengths."""

    def __init__(self, model, rows, pages, kind):
        self.model = model
        self.cache = q8.KVCache.empty(kind, LAYERS, pages, PAGE, KV, HEAD)
        self.table = torch.full((rows, 64), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")

    def prefill(self, rows, prompts):
        """Whole prompts [len, DIM] into empty rows: one packed forward pass."""
        lens = [p.shape[0] for p in prompts]
        q8.kv_reserve(self.cache, self.table, self.lens, self.refs, ints(rows), ints(lens))
        positions = torch.cat([torch.arange(n) for n in lens]).int().cuda()
        seq_of = torch.cat([torch.full((n,), r) for r, n in zip(rows, lens)]).int().cuda()
        start = ints([0, *torch.tensor(lens).cumsum(0).tolist()])

        def attend(layer, q, k, v):
            q, k, v = q8.kv_append(self.cache, layer, q, k, v, positions, seq_of, self.table, self.model.cos_sin, 1,
                                   torch.bfloat16, want_kv=True)
            return q8.attn_prompt(q, k, v, start, out_type=q8.Q8_TYPE_Q8_0)
        return self.model.forward(torch.cat(prompts), positions, attend)

    def step(self, rows, x):
        """One new token [len(rows), DIM] for each row."""
        idx = ints(rows)
        q8.kv_reserve(self.cache, self.table, self.lens, self.refs, idx, torch.ones_like(idx))
        at = idx.long()
        table, lens = self.table[at], self.lens[at]
        positions = lens - 1

        def attend(layer, q, k, v):
            q = q8.kv_append(self.cache, layer, q, k, v, positions, idx, self.table, self.model.cos_sin, 1, torch.bfloat16)
            return q8.attn_decode(q, self.cache, layer, table, lens, out_type=q8.Q8_TYPE_Q8_0)
        return self.model.forward(x, positions, attend)

    def fork(self, src, dst):
        q8.kv_fork(self.cache, self.table, self.lens, self.refs, ints(src), ints(dst))

    def free(self, rows):
        q8.kv_free(self.cache, self.table, self.lens, self.refs, ints(rows))

    def compact(self):
        self.table, self.refs, used = q8.kv_compact(self.cache, self.table, self.lens, self.refs)
        return int(used)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def whole(model, x):
    """The hidden states of one sequence without a cache."""
    n = x.shape[0]
    positions, start = torch.arange(n, dtype=torch.int32, device="cuda"), ints([0, n])

    def attend(layer, q, k, v):
        q, k, v = q8.kv_append(None, 0, q, k, v, positions, None, None, model.cos_sin, 1, torch.bfloat16, want_kv=True)
        return q8.attn_prompt(q, k, v, start, out_type=q8.Q8_TYPE_Q8_0)
    return model.forward(x, positions, attend)


def run(kind=q8.Q8_TYPE_BF16, steps=20):
    """-> the largest relative difference (2-norm) of a cached sequence's last hidden state from the whole one's."""
    model, g = Decoder(), torch.Generator(device="cuda").manual_seed(1)
    new = lambda n: torch.randn(n, DIM, generator=g, device="cuda")
    server = Server(model, rows=6, pages=64, kind=kind)
    history = {0: new(37), 1: new(5), 2: new(90)}
    server.prefill(list(history), list(history.values()))
    server.fork([0, 0], [3, 4])                       # two more branches of the first conversation
    for row in (3, 4):
        history[row] = history[0].clone()
    for i in range(steps):
        if i == steps // 2:                           # a branch ends; its pages go back, the pool closes up
            server.free([3])
            del history[3]
            server.compact()
        rows = list(history)
        x = new(len(rows))
        last = server.step(rows, x)
        for j, row in enumerate(rows):
            history[row] = torch.cat([history[row], x[j:j + 1]])
    assert q8.q8_last_error() == q8.Q8_OK
    worst = 0.0
    for j, row in enumerate(history):
        ref = whole(model, history[row])[-1]
        worst = max(worst, float((last[j] - ref).norm() / ref.norm()))
    return worst


if __name__ == "__main__":
    for name, kind in (("bf16", q8.Q8_TYPE_BF16), ("Q8_0", q8.Q8_TYPE_Q8_0)):
        print(f"{name} cache: cached and whole hidden states differ by {run(kind):.2e} (relative 2-norm)")
