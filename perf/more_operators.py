"""What a decoder layer that serves many requests needs around its Q8_0 projections and its paged cache, measured: the
cases, their plain forms in elementary torch operations, and the calls a user makes of the library for the same thing.

Operators (case["op"]):
  norm   the residual path between two blocks: the norm after a block, its gate, the scaled residual sum, the norm before
         the next block, written as Q8_0 blocks or as values
  lora   the low-rank adapters of many requests beside a shared projection: out = base + scale_a B_a (A_a x), a the
         token's adapter (negative: none)
  read   a paged cache's keys and values back as rows, for the attention of a prompt's next part

A Q8_0 block is 34 bytes: a binary16 scale and 32 int8.  A page of a cache holds, per key-value head, `page` rows of `dim`
values: 16 bit, or an int8 plane [page][dim] and a binary16 scale plane [page][dim / 32].
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "q8": 34 / 32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token between two blocks: a call that only latency bounds
        dict(name="norm one token", op="norm", tokens=1, dim=4096, h="f32", y="f32", out="q8", post=True, gate="row",
             scale=1.0),
        # a decoding batch whose residual stream is kept in 16 bit, gated per token
        dict(name="norm batch bf16", op="norm", tokens=48, dim=7168, h="bf16", y="bf16", out="q8", post=False,
             gate="token", scale=1.0),
        # a long prefill, fp32 stream into the next projection's blocks
        dict(name="norm prefill", op="norm", tokens=4096, dim=4096, h="f32", y="f32", out="q8", post=True, gate="row",
             scale=0.5),
        # a ragged batch of prompts of a narrower model, 16 bit in and out, gated per token
        dict(name="norm ragged bf16", op="norm", tokens=5003, dim=2080, h="bf16", y="f32", out="bf16", post=True,
             gate="token", scale=1.0),
        # one conversation with its adapter on a square projection: latency
        dict(name="lora one token", op="lora", tokens=1, ins=4096, outs=4096, rank=16, ragged=False, adapters=8,
             type="bf16", x="f32", requests=1, bare=0.0, shape=1),
        # a decoding batch, an adapter each, beside the wide projection, from the blocks that feed it
        dict(name="lora batch wide q8", op="lora", tokens=32, ins=1024, outs=32768, rank=32, ragged=True, adapters=40,
             type="bf16", x="q8", requests=32, bare=0.1, shape=2),
        # decoding and short prompts mixed, ranks of all sizes
        dict(name="lora mixed f16", op="lora", tokens=333, ins=2048, outs=1000, rank=64, ragged=True, adapters=12,
             type="f16", x="f32", requests=40, bare=0.2, shape=3),
        # the prompts of four requests packed together
        dict(name="lora prefill", op="lora", tokens=4096, ins=4096, outs=4096, rank=64, ragged=False, adapters=4,
             type="bf16", x="f32", requests=4, bare=0.0, shape=4),
        # the same beside the wide projection, from a 16-bit input
        dict(name="lora prefill wide", op="lora", tokens=2048, ins=1024, outs=32768, rank=16, ragged=True, adapters=6,
             type="bf16", x="bf16", requests=7, bare=0.0, shape=5),
        # the cached start of one conversation, for its next question
        dict(name="read one short", op="read", seqs=1, longest=300, kv=8, dim=128, type="bf16", out="bf16", page=64,
             first=0, shape=6),
        # prompts in parts over an 8-bit cache, the part that a window still sees
        dict(name="read parts q8", op="read", seqs=12, longest=8192, kv=8, dim=128, type="q8", out="bf16", page=64,
             first=1000, shape=7),
        # few long documents
        dict(name="read long f16", op="read", seqs=3, longest=60003, kv=4, dim=256, type="f16", out="f16", page=32,
             first=0, shape=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "lora", "lora", "lora", "read"])
    if op == "norm":
        dim = 32 * _log_int(rng, 4, 512)
        return dict(op=op, tokens=_log_int(rng, 1, max(2, min(16384, (1 << 24) // dim))), dim=dim,
                    h=rng.choice(["f32", "f32", "bf16", "f16"]), y=rng.choice(["f32", "f32", "bf16", "f16"]),
                    out=rng.choice(["q8", "q8", "f32", "bf16", "f16"]), post=rng.random() < 0.6,
                    gate=rng.choice(["none", "row", "token"]), scale=rng.choice([1.0, round(rng.uniform(0.1, 2.0), 3)]))
    shape = rng.randrange(1 << 30)
    if op == "lora":
        ins, outs, rank = 32 * _log_int(rng, 8, 256), _log_int(rng, 64, 32768), rng.choice([8, 16, 16, 32, 64, 128])
        adapters = _log_int(rng, 1, 64)
        adapters = max(1, min(adapters, (1 << 28) // (rank * (ins + outs))))
        # what the listed prefills cost: dense products over all adapters in the plain form, rows in and out in the kernel
        most = min(8192, (1 << 26) // max(ins, outs), 4 * 4096 * 64 * 8192 // (adapters * rank * (ins + outs)))
        tokens = _log_int(rng, 1, max(2, most))
        return dict(op=op, tokens=tokens, ins=ins, outs=outs, rank=rank, ragged=rng.random() < 0.6, adapters=adapters,
                    type=rng.choice(["bf16", "bf16", "f16"]), x=rng.choice(["f32", "f32", "q8", "bf16", "f16"]),
                    requests=rng.choice([1, tokens, max(1, min(tokens, _log_int(rng, 1, 64)))]),
                    bare=rng.choice([0.0, 0.0, 0.15, 0.5]), shape=shape)
    kv, dim, seqs = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256, 512]), _log_int(rng, 1, 32)
    longest = _log_int(rng, 1, max(2, min(60003, 150_000_000 // (seqs * kv * dim))))
    return dict(op=op, seqs=seqs, longest=longest, kv=kv, dim=dim, type=rng.choice(["q8", "q8", "bf16", "f16"]),
                out=rng.choice(["bf16", "f16", "f32"]), page=rng.choice([16, 32, 64, 128, 256]),
                first=rng.choice([0, 0, rng.randint(1, longest)]), shape=shape)


# ------------------------------------------------------------------ what a program has in hand
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device=DEV, dtype=torch.int32)


def _adapter_of(case):
    """Tokens' adapters on the host: the requests' tokens one after another, each request with one adapter or none."""
    r = np.random.RandomState(case["shape"] % (1 << 31))
    n, m = case["tokens"], case["requests"]
    cuts = np.sort(r.choice(n - 1, m - 1, replace=False)) + 1 if m > 1 else np.zeros(0, np.int64)
    ids = r.randint(0, case["adapters"], m)
    if m > 1:
        ids[r.uniform(size=m) < case["bare"]] = -1
    return np.repeat(ids, np.diff(np.concatenate([[0], cuts, [n]]).astype(np.int64)))


def _ranks(case):
    """The adapters' ranks: all the same, or of every size with the largest among them."""
    k = case["adapters"]
    if not case["ragged"]:
        return np.full(k, case["rank"])
    ranks = np.random.RandomState((case["shape"] + 1) % (1 << 31)).randint(1, case["rank"] + 1, k)
    ranks[0] = case["rank"]
    return ranks


def _spans(case):
    """First position and length of each sequence's part: lengths spread over their logarithm, one of them empty."""
    r = np.random.RandomState(case["shape"] % (1 << 31))
    n, top = case["seqs"], case["longest"]
    lens = np.exp(r.uniform(math.log(max(1, top / 32)), math.log(top + 0.5), n)).astype(np.int64).clip(1, top)
    lens[r.randint(n)] = top
    first = np.minimum(lens, case["first"]) if case["first"] else np.zeros(n, np.int64)
    first = np.where(lens == top, first // 2, first)
    return first, lens - first, lens


def _blocks(x):
    """fp32 rows -> the bytes of their Q8_0 blocks."""
    b = x.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1) / 127.0
    q = torch.where(d[..., None] > 0, torch.round(b / d.clamp(min=1e-30)[..., None]), 0.0).to(torch.int8)
    return torch.cat([d.half()[..., None].view(torch.uint8), q.view(torch.uint8)], -1).flatten(-2)


def _planes(pool):
    """16-bit rows [.., page, dim] -> the bytes of their Q8_0 planes."""
    x = pool.float().unflatten(-1, (-1, 32))
    d = x.abs().amax(-1) / 127.0
    q = torch.where(d[..., None] > 0, torch.round(x / d.clamp(min=1e-30)[..., None]), 0.0).to(torch.int8)
    return torch.cat([q.flatten(-3).view(torch.uint8), d.half().flatten(-2).view(torch.uint8)], -1)


def prepare(case, seed):
    g = _generator(seed)

    def normal(*shape, to=torch.float32):
        return torch.randn(shape, generator=g, device=DEV, dtype=to)

    s = {"case": case}
    if case["op"] == "norm":
        n, dim = case["tokens"], case["dim"]
        # a residual stream grows over the layers and has a few large channels; a block's output is smaller
        loud = 1.0 + 19.0 * (torch.rand(dim, generator=g, device=DEV) < 0.01)
        s["h"] = (3.0 * normal(n, dim) * loud).to(DTYPES[case["h"]])
        s["y"] = (0.3 * normal(n, dim)).to(DTYPES[case["y"]])
        s["post"] = 1.0 + 0.2 * normal(dim) if case["post"] else None
        s["next"] = 1.0 + 0.2 * normal(dim)
        s["gate"] = None if case["gate"] == "none" else 0.5 + 0.3 * normal(*([n] if case["gate"] == "token" else []), dim)
        s["dim"] = torch.full((), float(dim), device=DEV)
        s["step"] = torch.full((), 127.0, device=DEV)
    elif case["op"] == "lora":
        n, ins, outs, rank, dt = case["tokens"], case["ins"], case["outs"], case["rank"], DTYPES[case["type"]]
        x = normal(n, ins) * (1.0 + 19.0 * (torch.rand(n, ins, generator=g, device=DEV) < 0.01))
        s["x"] = _blocks(x) if case["x"] == "q8" else x.to(DTYPES[case["x"]])
        s["a"] = (normal(case["adapters"], rank, ins) * ins ** -0.5).to(dt)
        s["b"] = (normal(case["adapters"], outs, rank) * 0.05).to(dt)
        s["ids"], s["ranks"] = _ints(_adapter_of(case)), _ints(_ranks(case))
        s["scales"] = 16.0 / s["ranks"].float()
        s["base"] = normal(n, outs)
    else:
        kv, dim, page, dt = case["kv"], case["dim"], case["page"], torch.float16 if case["type"] == "f16" else torch.bfloat16
        first, count, lens = _spans(case)
        need = -(-lens // page)
        n_pages, width = int(need.sum()) + 3, int(need.max()) + 1
        order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        table, at = np.full((case["seqs"], width), -1, np.int64), 0
        for i, k in enumerate(need):
            table[i, :k] = np.arange(at, at + k)
            at += k
        t = torch.from_numpy(table).to(DEV)
        s["table"] = torch.where(t >= 0, order[t.clamp(min=0)], -1).to(torch.int32)
        s["first"], s["start"] = _ints(first), _ints(np.concatenate([[0], np.cumsum(count)]))
        s["rows"] = int(count.sum())
        for name in ("k", "v"):
            pool = normal(1, n_pages, kv, page, dim, to=dt)
            s[name] = _planes(pool).contiguous() if case["type"] == "q8" else pool
    return s


def work(case):
    if case["op"] == "norm":
        n, dim = case["tokens"], case["dim"]
        gate = {"none": 0, "row": dim, "token": n * dim}[case["gate"]]
        return {"bytes": n * dim * (2 * BYTES[case["h"]] + BYTES[case["y"]] + BYTES[case["out"]]) + 4 * (gate + 2 * dim),
                "flops": 8 * n * dim}
    if case["op"] == "lora":
        ids, ranks = _adapter_of(case), _ranks(case)
        used = int(ranks[np.unique(ids[ids >= 0])].sum())
        live = int(ranks[ids[ids >= 0]].sum())
        both = case["ins"] + case["outs"]
        return {"bytes": int((ids >= 0).sum()) * case["ins"] * BYTES[case["x"]] + case["tokens"] * case["outs"] * 8
                + used * both * 2 + case["tokens"] * 4, "flops": 2 * live * both}
    _, count, _ = _spans(case)
    values = int(count.sum()) * case["kv"] * case["dim"] * 2
    return {"bytes": values * (BYTES[case["type"]] + BYTES[case["out"]]), "flops": 0}


# ------------------------------------------------------------------ plain forms
def _inverse_rms(x, dim):
    """1 / sqrt(mean x^2 + eps) of fp32 rows, every step rounded to fp32 once."""
    total = x.double().square().sum(-1, keepdim=True).float()
    return ((total / dim) + EPS).sqrt().reciprocal()


def _plain_norm(s):
    case = s["case"]
    h, u = s["h"].float(), s["y"].float()
    if case["post"]:
        u = u * _inverse_rms(u, s["dim"]) * s["post"]
    if s["gate"] is not None:
        u = s["gate"] * u
    stored = (case["scale"] * h + u).to(s["h"].dtype)
    h = stored.float()
    y = h * _inverse_rms(h, s["dim"]) * s["next"]
    if case["out"] != "q8":
        return {"h": stored, "n": y.to(DTYPES[case["out"]])}
    b = y.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / s["step"]
    z = torch.where(d > 0, b / d, 0.0)
    q = torch.trunc(z)
    q = q + torch.where((z - q).abs() >= 0.5, torch.sign(z), 0.0)      # halves away from zero
    return {"h": stored, "d": d[..., 0].half(), "q": q.to(torch.int8)}


def _values(blocks):
    """Q8_0 blocks -> the values they stand for, in fp32."""
    b = blocks.unflatten(-1, (-1, 34))
    return (b[..., 2:].contiguous().view(torch.int8).float() * b[..., :2].contiguous().view(torch.float16).float()).flatten(-2)


def _plain_lora(s):
    x = _values(s["x"]) if s["case"]["x"] == "q8" else s["x"].float()
    a, b = s["a"].float(), s["b"].float()
    k, rank, _ = a.shape
    # every adapter's products, and of them each token's own
    mine = s["ids"][:, None] == torch.arange(k, device=DEV)
    rows = torch.arange(rank, device=DEV) < s["ranks"][:, None]
    seen = (mine[:, :, None] & rows) * s["scales"][:, None]
    low = (x @ a.flatten(0, 1).T).unflatten(1, (k, rank)) * seen
    return s["base"] + low.flatten(1) @ b.transpose(1, 2).flatten(0, 1)


def _plain_read(s):
    case = s["case"]
    page, dim = case["page"], case["dim"]
    i = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(s["start"].long(), i, right=True) - 1
    pos = i - s["start"][seq] + s["first"][seq]
    at, row = s["table"][seq, pos // page].long()[:, None], (pos % page)[:, None]
    head = torch.arange(case["kv"], device=DEV)
    out = []
    for pool in (s["k"][0], s["v"][0]):
        if case["type"] == "q8":
            q = pool[..., :page * dim].view(torch.int8).unflatten(-1, (page, dim))[at, head, row]
            d = pool[..., page * dim:].unflatten(-1, (page, dim // 16))[at, head, row].view(torch.float16)
            x = (q.unflatten(-1, (-1, 32)).float() * d.float()[..., None]).flatten(-2)
        else:
            x = pool[at, head, row].float()
        out.append(x.to(DTYPES[case["out"]]))
    return {"k": out[0], "v": out[1]}


PLAIN = {"norm": _plain_norm, "lora": _plain_lora, "read": _plain_read}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import q8_quantized_matmul_gb300 as q8
    case = s["case"]
    kinds = {"f32": q8.Q8_TYPE_F32, "f16": q8.Q8_TYPE_F16, "bf16": q8.Q8_TYPE_BF16, "q8": q8.Q8_TYPE_Q8_0}
    if case["op"] == "norm":
        n, h = q8.residual_norm(s["h"], s["y"], s["next"], EPS, gamma_post=s["post"], post=case["post"], gate=s["gate"],
                                residual_scale=case["scale"], out_type=kinds[case["out"]])
        if case["out"] != "q8":
            return {"h": h, "n": n}
        # a block's scale and whole numbers, where they lie
        n = n.view(case["tokens"], -1, 34)
        return {"h": h, "d": n[..., :2].view(torch.float16)[..., 0], "q": n[..., 2:].view(torch.int8)}
    if case["op"] == "lora":
        return q8.lora(s["x"], s["a"], s["b"], s["ids"], ranks=s["ranks"], scales=s["scales"], base=s["base"])
    cache = q8.KVCache(s["k"], s["v"], kinds[case["type"]], case["page"], case["kv"], case["dim"])
    k, v = q8.kv_read(cache, 0, s["table"], s["start"], s["rows"], first=s["first"], out_type=kinds[case["out"]])
    return {"k": k, "v": v}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_norm(case, s):
    def normalised(x, gamma):
        return x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * gamma.double()
    u = s["y"].double()
    if case["post"]:
        u = normalised(u, s["post"])
    gate = 1.0 if s["gate"] is None else s["gate"].double()
    h = s["h"].double() * case["scale"] + u * gate
    n = normalised(h, s["next"])
    if case["out"] != "q8":
        return {"h": h, "n": n}
    return {"h": h, "d": n.view(case["tokens"], -1, 32).abs().amax(2) / 127, "q": None}


def _exact_lora(case, s):
    if case["x"] == "q8":
        raw = s["x"].view(case["tokens"], -1, 34)
        x = raw[:, :, 2:].contiguous().view(torch.int8).double() * raw[:, :, :2].contiguous().view(torch.float16).double()
        x = x.view(case["tokens"], case["ins"])
    else:
        x = s["x"].double()
    out = s["base"].double()
    ids, ranks = _adapter_of(case), _ranks(case)
    for k in np.unique(ids[ids >= 0]):
        t = torch.from_numpy(np.flatnonzero(ids == k)).to(DEV)
        r = int(ranks[k])
        low = x[t] @ s["a"][k, :r].double().T
        out[t] += (low @ s["b"][k, :, :r].double().T) * (16.0 / r)
    return out


def _exact_read(case, s):
    first, count, _ = _spans(case)
    page, dim = case["page"], case["dim"]
    both = {"k": [], "v": []}
    for name, parts in both.items():
        for i in range(case["seqs"]):
            at = s["table"][i, first[i] // page:-(-(first[i] + count[i]) // page)].long()
            x = s[name][0][at]
            if case["type"] == "q8":
                d = x[..., page * dim:].contiguous().view(torch.float16).double()
                x = x[..., :page * dim].contiguous().view(torch.int8).double()
                x = (x.view(*x.shape[:-1], -1, 32) * d[..., None]).view(*x.shape[:-1], page, dim)
            x = x.double().transpose(1, 2).reshape(-1, case["kv"], dim)
            parts.append(x[first[i] % page:first[i] % page + count[i]])
    return {name: torch.cat(parts) for name, parts in both.items()}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "lora": _exact_lora, "read": _exact_read}[case["op"]](case, s)
