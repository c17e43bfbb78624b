"""The paged key-value cache and the attention over it, measured: the cases, their plain forms in
elementary torch operations, and the calls a user makes of the library for the same thing.

A cache holds, per layer, pages of `page` tokens; a page holds, per key-value head, `page` rows of
`dim` values: 16-bit values, or Q8_0 as an int8 plane [page][dim] followed by a binary16 scale plane
[page][dim / 32].  A table row lists a sequence's pages; `refs` counts how many table rows hold a page.

Operators (case["op"]):
  append   rotate new tokens' q and k, round q, store k and v in the pages
  decode   one new token per sequence attends to its cached tokens
  prompt   every token of packed sequences attends to the keys up to its own
  fork     release the rows of finished branches, then fork running sequences into them
  compact  move the pages in use to the front of the pool
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
NEG = -math.inf


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the first answer tokens of one conversation: a call that only latency bounds
        dict(name="decode one short", op="decode", seqs=1, longest=300, heads=32, kv=8, dim=128, type="bf16", page=64,
             window=0, sinks=False, shape=1),
        # a serving batch: conversations of very different lengths, one just opened (no token cached yet)
        dict(name="decode ragged batch", op="decode", seqs=48, longest=16000, heads=32, kv=8, dim=128, type="bf16",
             page=64, window=0, sinks=False, shape=2),
        # few long documents over the 8-bit cache
        dict(name="decode long q8", op="decode", seqs=4, longest=100003, heads=64, kv=8, dim=128, type="q8", page=128,
             window=0, sinks=False, shape=3),
        # the 64 heads of 512 that q_b projects to, all on one key-value head, with sinks
        dict(name="decode 64x512 shared", op="decode", seqs=16, longest=4100, heads=64, kv=1, dim=512, type="f16",
             page=32, window=0, sinks=True, shape=4),
        # a short question: latency
        dict(name="prompt one short", op="prompt", seqs=1, longest=77, prefix=0, heads=32, kv=8, dim=128, type="bf16",
             window=0, sinks=False, shape=5),
        # prompts of different lengths packed together, after cached prefixes, in a sliding window
        dict(name="prompt packed window", op="prompt", seqs=12, longest=2048, prefix=500, heads=32, kv=4, dim=64,
             type="f16", window=1024, sinks=True, shape=6),
        # one long document
        dict(name="prompt long", op="prompt", seqs=1, longest=8192, prefix=0, heads=32, kv=8, dim=128, type="bf16",
             window=0, sinks=False, shape=7),
        # one decode step's new tokens into the 8-bit cache
        dict(name="append step q8", op="append", seqs=32, longest=1, heads=32, kv=8, dim=128, type="q8", page=64,
             rope=1, rot=128, shape=8),
        # the 4096 tokens of a long prefill into a 16-bit cache
        dict(name="append prefill", op="append", seqs=4, longest=1024, heads=32, kv=8, dim=128, type="bf16", page=64,
             rope=2, rot=64, shape=9),
        # a beam step of one request over a small cache
        dict(name="fork few", op="fork", seqs=4, longest=700, branches=4, pages=256, layers=2, kv=8, dim=128,
             type="bf16", page=16, shape=10),
        # parallel samples of many requests over all layers
        dict(name="fork many", op="fork", seqs=32, longest=500, branches=3, pages=1024, layers=16, kv=4, dim=64,
             type="bf16", page=32, shape=11),
        # defragmenting a half-empty pool after a burst
        dict(name="compact pool", op="compact", seqs=64, longest=300, branches=1, pages=1200, layers=16, kv=4, dim=64,
             type="bf16", page=32, shape=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "prompt", "prompt", "prompt", "append", "append", "fork", "compact"])
    shape = rng.randrange(1 << 30)
    if op == "decode":
        kv, group, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8, 12, 16]), rng.choice([64, 128, 128])
        if rng.random() < 0.2:
            kv, group, dim = 1, 64, 512
        seqs = _log_int(rng, 1, 64)
        most = 4_000_000 // (seqs * kv * dim // 64)   # keeps the cached values under the largest listed case's
        return dict(op=op, seqs=seqs, longest=_log_int(rng, 1, max(2, min(100003, most))), heads=kv * group, kv=kv,
                    dim=dim, type=rng.choice(["bf16", "f16", "q8"]), page=rng.choice([16, 32, 64, 128]),
                    window=rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]), sinks=rng.random() < 0.4, shape=shape)
    if op == "prompt":
        kv, group, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8]), rng.choice([64, 128, 128])
        if rng.random() < 0.15:
            kv, group, dim = 1, rng.choice([16, 64]), 512
        seqs, heads = _log_int(rng, 1, 16), kv * group
        prefix = rng.choice([0, 0, _log_int(rng, 1, 1000)])
        most = math.isqrt(int(32 * 8192 * 8192 * 128 // (heads * dim * seqs)))   # the padded scores of the largest case
        return dict(op=op, seqs=seqs, longest=_log_int(rng, 1, max(2, min(8192, most - prefix))), prefix=prefix,
                    heads=heads, kv=kv, dim=dim, type=rng.choice(["bf16", "f16"]),
                    window=rng.choice([0, 0, _log_int(rng, 1, 4096)]), sinks=rng.random() < 0.4, shape=shape)
    if op == "append":
        kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        rope = rng.choice([0, 1, 2])
        return dict(op=op, seqs=_log_int(rng, 1, 64), longest=_log_int(rng, 1, 128), heads=kv * rng.choice([1, 2, 4, 5]),
                    kv=kv, dim=dim, type=rng.choice(["bf16", "f16", "q8"]), page=rng.choice([16, 32, 64, 128]),
                    rope=rope, rot=rng.choice([32, 64, dim]) if rope else 0, shape=shape)
    seqs, page = _log_int(rng, 2, 32), rng.choice([16, 32, 64])
    branches = rng.randint(1, 3) if op == "fork" else 1
    longest = _log_int(rng, 2, 400)
    pages = seqs * (branches + 1) * (-(-longest // page)) + rng.randint(8, 128)
    return dict(op=op, seqs=seqs, longest=longest, branches=branches, pages=pages, layers=rng.randint(1, 4),
                kv=rng.choice([1, 2, 4]), dim=rng.choice([64, 128]), type="bf16", page=page, shape=shape)


def _lens(case, empty):
    """The sequences' lengths: the longest one, one empty where there may be one, the others spread over their logarithm."""
    r = np.random.RandomState(case["shape"] % (1 << 31))
    n, top = case["seqs"], case["longest"]
    lens = np.exp(r.uniform(math.log(max(1, top / 32)), math.log(top + 0.5), n)).astype(np.int64).clip(1, top)
    lens[r.randint(n)] = top
    if empty and n > 2 and lens[1] != top:
        lens[1] = 0
    return lens


def _bytes_per_value(case):
    return 34 / 32 if case["type"] == "q8" else 2


def _pairs(case):
    """(query, key) pairs that one head of a prompt case computes."""
    total = 0
    for n in _lens(case, False):
        last = np.arange(n, dtype=np.int64) + case["prefix"] + 1
        total += int((np.minimum(last, case["window"]) if case["window"] else last).sum())
    return total


def work(case):
    op, kv, dim = case["op"], case["kv"], case["dim"]
    if op == "decode":
        lens = _lens(case, True)
        seen = int((np.minimum(lens, case["window"]) if case["window"] else lens).sum())
        qo = case["seqs"] * case["heads"] * dim * 2 * 2
        return {"bytes": seen * kv * dim * 2 * _bytes_per_value(case) + qo, "flops": 4 * seen * case["heads"] * dim}
    if op == "prompt":
        n = int(_lens(case, False).sum())
        nk = n + case["prefix"] * case["seqs"]
        return {"bytes": 2 * (2 * n * case["heads"] + 2 * nk * kv) * dim, "flops": 4 * _pairs(case) * case["heads"] * dim}
    if op == "append":
        n = int(_lens(case, False).sum())
        vals = n * kv * dim * 2
        return {"bytes": n * case["heads"] * dim * 6 + vals * (4 + _bytes_per_value(case)),
                "flops": 3 * n * (case["heads"] + kv) * case.get("rot", 0)}
    lens, page = _lens(case, False), case["page"]
    page_bytes = case["layers"] * 2 * kv * dim * 2 * page
    if op == "fork":
        moved = int((lens % page != 0).sum()) * case["branches"]
    else:
        refs = _layout(case)[2]
        moved = int((refs[int((refs > 0).sum()):] > 0).sum())
    return {"bytes": 2 * moved * page_bytes + 8 * int((-(-lens // page)).sum()) + 8 * case["pages"], "flops": 0}


# ------------------------------------------------------------------ what a program has in hand
def _dtype(case):
    return torch.bfloat16 if case["type"] == "bf16" else torch.float16


def _layout(case):
    """Table, lengths and reference counts on the host: pages handed out in a scattered order."""
    r = np.random.RandomState((case["shape"] + 1) % (1 << 31))
    lens, page, n = _lens(case, False), case["page"], case["seqs"]
    rows = n * (case["branches"] + 1) if case["op"] == "fork" else n
    width = -(-case["longest"] // page) + 1
    table = np.full((rows, width), -1, np.int32)
    refs = np.zeros(case["pages"], np.int32)
    order, at = r.permutation(case["pages"]), 0
    for i, k in enumerate(-(-lens // page)):
        table[i, :k] = order[at:at + k]
        at += k
    refs[order[:at]] = 1
    all_lens = np.zeros(rows, np.int32)
    all_lens[:n] = lens
    return table, all_lens, refs


def _quantised(pool):
    """16-bit rows [.., page, dim] -> the bytes of their Q8_0 planes [.., page * dim + page * dim / 32 * 2]."""
    x = pool.float().unflatten(-1, (-1, 32))
    d = x.abs().amax(-1) / 127.0
    q = torch.where(d[..., None] > 0, torch.round(x / d.clamp(min=1e-30)[..., None]), 0.0).to(torch.int8)
    return torch.cat([q.flatten(-3).view(torch.uint8), d.half().flatten(-2).view(torch.uint8)], -1)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, kv, dim, dt = case["op"], case["kv"], case["dim"], _dtype(case)

    def normal(*shape, to=None):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32 if to is None else to)

    def ints(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(device=DEV, dtype=torch.int32)

    s = {"case": case}
    if op == "decode":
        lens = _lens(case, True)
        need = -(-lens // case["page"])
        n_pages, width = int(need.sum()) + 3, int(need.max()) + 1
        order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
        table, at = np.full((case["seqs"], width), -1, np.int64), 0
        for i, k in enumerate(need):
            table[i, :k] = np.arange(at, at + k)
            at += k
        t = torch.from_numpy(table).to(DEV)
        s["table"] = torch.where(t >= 0, order[t.clamp(min=0)], -1).to(torch.int32)
        s["lens"] = ints(lens)
        for name in ("k", "v"):
            pool = normal(1, n_pages, kv, case["page"], dim, to=dt)
            s[name] = _quantised(pool).contiguous() if case["type"] == "q8" else pool
        s["q"] = normal(case["seqs"], case["heads"], dim).to(dt)
        s["sinks"] = normal(case["heads"]) if case["sinks"] else None
    elif op == "prompt":
        lens = _lens(case, False)
        start = np.concatenate([[0], np.cumsum(lens)])
        kstart = start + np.arange(len(start)) * case["prefix"]
        s["q_start"], s["k_start"] = ints(start), ints(kstart)
        s["q"] = normal(int(start[-1]), case["heads"], dim, to=dt)
        # k and v side by side, as one projection writes them
        both = normal(int(kstart[-1]), 2 * kv, dim, to=dt)
        s["k"], s["v"] = both[:, :kv], both[:, kv:]
        s["sinks"] = normal(case["heads"]) if case["sinks"] else None
    elif op == "append":
        lens = _lens(case, False)
        n, page = int(lens.sum()), case["page"]
        had = np.random.RandomState((case["shape"] + 2) % (1 << 31)).randint(0, 2000, case["seqs"])
        need = -(-(had + lens) // page)
        n_pages = int(need.sum()) + 2
        perm = np.random.RandomState((case["shape"] + 3) % (1 << 31)).permutation(n_pages)
        table, at = np.full((case["seqs"], int(need.max())), -1, np.int32), 0
        for i, k in enumerate(need):
            table[i, :k] = perm[at:at + k]
            at += k
        s["table"] = ints(table)
        s["seq_of"] = ints(np.repeat(np.arange(case["seqs"]), lens))
        s["positions"] = ints(np.concatenate([np.arange(h, h + m) for h, m in zip(had, lens)]))
        row = page * dim if case["type"] != "q8" else page * dim + page * dim // 16
        for name in ("k", "v"):
            s[name + "_pool"] = torch.zeros(1, n_pages, kv, row, device=DEV,
                                            dtype=torch.uint8 if case["type"] == "q8" else dt)
        qkv = normal(n, (case["heads"] + 2 * kv) * dim)
        q, k, v = qkv.split([case["heads"] * dim, kv * dim, kv * dim], 1)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, dim)) for x in (q, k, v))
        if case["rope"]:
            half = case["rot"] // 2
            f = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
            a = torch.arange(int((had + lens).max()) + 1, device=DEV, dtype=torch.float64)[:, None] * f
            s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
        else:
            s["cos_sin"] = None
    else:
        table, lens, refs = _layout(case)
        s["table"], s["lens"], s["refs"] = ints(table), ints(lens), ints(refs)
        for name in ("k", "v"):
            s[name] = normal(case["layers"], case["pages"], kv, case["page"], dim, to=dt)
        n, b = case["seqs"], case["branches"]
        if op == "fork":
            s["src"] = ints(np.repeat(np.arange(n), b))
            s["dst"] = ints(n + np.arange(n * b))
    return s


# ------------------------------------------------------------------ plain forms
def _values(pool, page, dim):
    """Q8_0 planes -> the values they stand for, in fp32."""
    q = pool[..., :page * dim].contiguous().view(torch.int8).unflatten(-1, (page, -1, 32)).float()
    d = pool[..., page * dim:].contiguous().view(torch.float16).unflatten(-1, (page, -1)).float()
    return (q * d[..., None]).flatten(-2)


def _softmax_product(s, seen, v, sinks):
    """s [.., heads, rows, keys] masked by seen [.., 1, rows, keys]; sinks [.., heads, 1, 1] or None; v [.., heads, keys, dim]."""
    s = s.masked_fill(~seen, NEG)
    m = s.amax(-1, keepdim=True)
    if sinks is not None:
        m = torch.maximum(m, sinks)
    m = torch.where(m == NEG, 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    if sinks is not None:
        total = total + torch.exp(sinks - m)
    return (p @ v) / torch.where(total == 0, 1.0, total)


def _plain_decode(s):
    case = s["case"]
    n, kv, dim, heads, page = case["seqs"], case["kv"], case["dim"], case["heads"], case["page"]
    at = s["table"].long().clamp(min=0)
    k, v = s["k"][0][at], s["v"][0][at]                       # [n, pages, kv, page, dim]
    k, v = (_values(x, page, dim) if case["type"] == "q8" else x.float() for x in (k, v))
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))  # [n, kv, tokens, dim]
    j = torch.arange(k.shape[2], device=DEV)
    seen = j < s["lens"][:, None]
    if case["window"]:
        seen = seen & (j >= s["lens"][:, None] - case["window"])
    v = torch.where(seen[:, None, :, None], v, 0.0)
    q = s["q"].float().view(n, kv, heads // kv, dim)
    sinks = None if s["sinks"] is None else s["sinks"].view(1, kv, heads // kv, 1)
    o = _softmax_product((q @ k.transpose(2, 3)) / math.sqrt(dim), seen[:, None, None], v, sinks)
    return o.reshape(n, heads, dim).to(s["q"].dtype)


def _plain_prompt(s):
    case = s["case"]
    n, kv, dim, heads, dt = case["seqs"], case["kv"], case["dim"], case["heads"], s["q"].dtype
    longest, group = case["longest"], case["heads"] // case["kv"]
    i = torch.arange(longest, device=DEV)
    j = torch.arange(longest + case["prefix"], device=DEV)
    q0, k0 = s["q_start"].long(), s["k_start"].long()
    ql, kl = q0.diff(), k0.diff()
    q = s["q"][(q0[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)].float()
    at = (k0[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    inside = j < kl[:, None]
    k, v = s["k"][at].float(), torch.where(inside[:, :, None, None], s["v"][at].float(), 0.0)
    q = q.view(n, longest, kv, group, dim).permute(0, 2, 3, 1, 4)              # [n, kv, group, rows, dim]
    k, v = k.permute(0, 2, 1, 3).unsqueeze(2), v.permute(0, 2, 1, 3).unsqueeze(2)
    last = i + (kl - ql)[:, None]                                              # [n, rows]
    seen = (j <= last[..., None]) & inside[:, None]
    if case["window"]:
        seen = seen & (j > last[..., None] - case["window"])
    sinks = None if s["sinks"] is None else s["sinks"].view(1, kv, group, 1, 1)
    o = _softmax_product((q @ k.transpose(3, 4)) / math.sqrt(dim), seen[:, None, None], v, sinks)
    t = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(q0, t, right=True) - 1
    return o.permute(0, 3, 1, 2, 4)[seq, t - q0[seq]].reshape(-1, heads, dim).to(dt)


def _rotated(x, cs, mode):
    if cs is None:
        return x
    rot = cs.shape[1]
    c, sn = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if mode == 1 else (x[..., 0:rot:2], x[..., 1:rot:2])
    a, b = a * c - b * sn, b * c + a * sn
    head = torch.cat([a, b], -1) if mode == 1 else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([head, x[..., rot:]], -1)


def _plain_append(s):
    case = s["case"]
    kv, dim, page = case["kv"], case["dim"], case["page"]
    cs = None if s["cos_sin"] is None else s["cos_sin"][s["positions"].long()]
    q, k = _rotated(s["q"], cs, case["rope"]), _rotated(s["k"], cs, case["rope"])
    pos = s["positions"].long()
    at = s["table"][s["seq_of"].long(), pos // page].long()
    row = (pos % page)[:, None]
    h = torch.arange(kv, device=DEV)
    for x, pool in ((k, s["k_pool"][0]), (s["v"], s["v_pool"][0])):
        if case["type"] == "q8":
            b = x.unflatten(-1, (-1, 32))
            d = b.abs().amax(-1, keepdim=True) / 127.0
            y = torch.where(d > 0, b / d, 0.0)
            r = torch.trunc(y)
            r = r + torch.where((y - r).abs() >= 0.5, torch.sign(y), 0.0)      # halves away from zero
            quants = pool[..., :page * dim].unflatten(-1, (page, dim))
            scales = pool[..., page * dim:].unflatten(-1, (page, dim // 16))
            quants[at[:, None], h, row] = r.to(torch.int8).flatten(-2).view(torch.uint8)
            scales[at[:, None], h, row] = d[..., 0].half().view(torch.uint8)
        else:
            pool.unflatten(-1, (page, dim))[at[:, None], h, row] = x.to(pool.dtype)
    return {"q": q.to(_dtype(case)), "k": s["k_pool"], "v": s["v_pool"]}


def _plain_fork(s):
    case = s["case"]
    page, refs, table, lens = case["page"], s["refs"], s["table"], s["lens"]
    src, dst = s["src"].long(), s["dst"].long()
    slot = torch.arange(table.shape[1], device=DEV)
    # release
    held = table[dst]
    live = slot < (lens[dst][:, None] + page - 1) // page
    refs.index_add_(0, held.clamp(min=0).flatten().long(), -live.int().flatten())
    # fork: whole pages shared, a part-filled last page copied to the lowest free page
    n = lens[src]
    whole, part = n // page, n % page != 0
    free = torch.sort(refs != 0, stable=True)[1]
    fresh = free[(torch.cumsum(part, 0) - part.int()).clamp(max=free.numel() - 1)]
    rows = table[src]
    last = rows.gather(1, whole[:, None].long())[:, 0]
    shared = slot < whole[:, None]
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), shared.int().flatten())
    refs.index_add_(0, fresh, part.int())
    tail = (slot == whole[:, None]) & part[:, None]
    table[dst] = torch.where(shared, rows, torch.where(tail, fresh[:, None].int(), -1)).int()
    lens[dst] = n
    moved = part.nonzero()[:, 0]
    to, fr = fresh[moved], last[moved].long()
    for pool in (s["k"], s["v"]):
        pool[:, to] = pool[:, fr]
    return {"table": table, "lens": lens, "refs": refs, "k": s["k"], "v": s["v"]}


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    used = refs > 0
    count = used.sum()
    at = torch.arange(refs.numel(), device=DEV)
    holes = (~used & (at < count)).nonzero()[:, 0]
    movers = (used & (at >= count)).nonzero()[:, 0]
    to = at.clone()
    to[movers] = holes
    new_refs = torch.where(at < count, refs, 0)
    new_refs[holes] = refs[movers]
    new_table = torch.where(table >= 0, to[table.clamp(min=0).long()].int(), -1)
    for pool in (s["k"], s["v"]):
        pool[:, holes] = pool[:, movers]
    return {"table": new_table, "refs": new_refs, "used": count.int(), "k": s["k"], "v": s["v"]}


PLAIN = {"decode": _plain_decode, "prompt": _plain_prompt, "append": _plain_append, "fork": _plain_fork,
         "compact": _plain_compact}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    import q8_quantized_matmul_gb300 as q8
    case = s["case"]
    op = case["op"]
    if op == "prompt":
        return q8.attn_prompt(s["q"], s["k"], s["v"], s["q_start"], s["k_start"], window=case["window"],
                              sinks=s["sinks"])
    k, v = (s["k_pool"], s["v_pool"]) if op == "append" else (s["k"], s["v"])
    kind = {"q8": q8.Q8_TYPE_Q8_0, "f16": q8.Q8_TYPE_F16, "bf16": q8.Q8_TYPE_BF16}[case["type"]]
    cache = q8.KVCache(k, v, kind, case["page"], case["kv"], case["dim"])
    if op == "decode":
        return q8.attn_decode(s["q"], cache, 0, s["table"], s["lens"], window=case["window"], sinks=s["sinks"])
    if op == "append":
        q = q8.kv_append(cache, 0, s["q"], s["k"], s["v"], s["positions"], s["seq_of"], s["table"],
                         cos_sin=s["cos_sin"], rope=case["rope"], dtype=_dtype(case))
        return {"q": q, "k": s["k_pool"], "v": s["v_pool"]}
    if op == "fork":
        q8.kv_free(cache, s["table"], s["lens"], s["refs"], s["dst"])
        q8.kv_fork(cache, s["table"], s["lens"], s["refs"], s["src"], s["dst"])
        return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], "k": s["k"], "v": s["v"]}
    table, refs, used = q8.kv_compact(cache, s["table"], s["lens"], s["refs"])
    return {"table": table, "refs": refs, "used": used, "k": s["k"], "v": s["v"]}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_rows(q, k, v, last, window, sinks):
    """q [rows, heads, dim], k and v [keys, kv, dim], last [rows]: the newest key each row sees."""
    rows, heads, dim = q.shape
    group = heads // k.shape[1]
    out = torch.zeros(rows, heads, dim, dtype=torch.float64, device=q.device)
    if k.shape[0] == 0:
        return out
    j = torch.arange(k.shape[0], device=q.device)
    for r0 in range(0, rows, 1024):
        la = last[r0:r0 + 1024, None]
        see = j <= la
        if window:
            see = see & (j > la - window)
        for h in range(heads):
            z = (q[r0:r0 + 1024, h].double() @ k[:, h // group].double().T) * dim ** -0.5
            z = torch.where(see, z, NEG)
            if sinks is not None:
                z = torch.cat([z, sinks[h].double().expand(z.shape[0], 1)], 1)
            w = torch.softmax(z, 1)[:, :k.shape[0]]
            w = torch.where(see.any(1, keepdim=True), w, 0.0)
            out[r0:r0 + 1024, h] = w @ v[:, h // group].double()
    return out


def exact(case, seed):
    op, dim, kv = case["op"], case["dim"], case["kv"]
    w = work(case)
    if op in ("fork", "compact") or w["flops"] > 6e11:
        return None
    s = prepare(case, seed)
    if op == "prompt":
        q0, k0 = s["q_start"].tolist(), s["k_start"].tolist()
        parts = []
        for a in range(case["seqs"]):
            q, k, v = s["q"][q0[a]:q0[a + 1]], s["k"][k0[a]:k0[a + 1]], s["v"][k0[a]:k0[a + 1]]
            last = torch.arange(q.shape[0], device=DEV) + k.shape[0] - q.shape[0]
            parts.append(_exact_rows(q, k, v, last, case["window"], s["sinks"]))
        return torch.cat(parts)
    if op == "decode":
        parts, page = [], case["page"]
        for a, n in enumerate(s["lens"].tolist()):
            if n == 0:
                parts.append(torch.zeros(1, case["heads"], dim, dtype=torch.float64, device=DEV))
                continue
            at = s["table"][a, :-(-n // page)].long()
            kv_rows = []
            for pool in (s["k"][0][at], s["v"][0][at]):
                if case["type"] == "q8":
                    d = pool[..., page * dim:].contiguous().view(torch.float16).double()
                    x = pool[..., :page * dim].contiguous().view(torch.int8).double()
                    pool = (x.view(*x.shape[:-1], -1, 32) * d[..., None]).view(*x.shape[:-1], page, dim)
                kv_rows.append(pool.transpose(1, 2).reshape(-1, kv, dim)[:n])
            last = torch.full((1,), n - 1, device=DEV)
            parts.append(_exact_rows(s["q"][a:a + 1], *kv_rows, last, case["window"], s["sinks"]))
        return torch.cat(parts)
    q = s["q"].double().clone()
    if case["rope"]:
        half = case["rot"] // 2
        cs = s["cos_sin"][s["positions"].long()].double()
        even = torch.arange(half, device=DEV)
        a, b = (even, even + half) if case["rope"] == 1 else (2 * even, 2 * even + 1)
        x, y, c, sn = q[..., a], q[..., b], cs[:, None, :half], cs[:, None, half:]
        q[..., a], q[..., b] = x * c - y * sn, x * sn + y * c
    return {"q": q, "k": None, "v": None}
