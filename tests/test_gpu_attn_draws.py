"""GPU tests of q8_attn_decode and q8_attn_prompt on drawn cases: formats, head layouts, page sizes, lengths from none to
thousands, windows, sinks, layers and strides in all combinations, against the definition in 64 bits on the GPU with the
error terms of tests/attn_plain.py.  What no query may see is NaN or infinite in the caches and behind the keys."""
import math
import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module")
def q8():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_quantized_matmul_gb300 import build
    build.build()
    import q8_quantized_matmul_gb300 as m
    torch.cuda.set_device(0)
    return m


def compare(out, lse, q, k, v, see, scale, sinks, weights, what):
    """out and lse (fp32 results) of q [heads, rows, D] over k and v [heads, keys, D], all float64; see [rows, keys]."""
    heads, rows, d = q.shape
    n = k.shape[1]
    z = torch.where(see, (q @ k.transpose(1, 2)) * scale, -math.inf)
    size = (d + 8) * 2.0 ** -23 * scale * (q.abs() @ k.abs().transpose(1, 2)) + 4 * z.abs() * 2.0 ** -23
    extra = torch.full((heads, rows, 1), -math.inf, dtype=torch.float64, device=DEV) if sinks is None else sinks[:, None, None].expand(-1, rows, 1)
    full = torch.logsumexp(torch.cat([z, extra], -1), -1)
    w = torch.exp(z - torch.where(full.isinf(), 0.0, full)[..., None]) * ~full.isinf()[..., None]
    ref, mean = w @ v, w @ v.abs()
    dz = torch.where(see, size, 0.0).amax(-1) if n else torch.zeros_like(full)
    seen = see.sum(-1)
    sums = 2.0 ** -21 + (seen / 8 + 16) * 2.0 ** -23
    bound = mean * (HALF_STEP[weights] + 2 * dz[..., None] + sums[:, None]) + 2.0 ** -24 * ref.abs() + 1e-30
    if weights == "f16" and n:
        bound = bound + 2.0 ** -24 * seen[None, :, None] * v.abs().amax(1, keepdim=True)
    err = (out - ref).abs()
    assert bool((err <= bound).all()), f"{what}: {float((err / bound).max()):.2f} of the bound"     # NaN fails too
    inf = full.isinf()
    assert torch.equal(lse[inf], full[inf]), f"{what}: infinite lse"
    assert bool(((lse - full).abs() <= 2 * dz + sums + 8 * full.abs() * 2.0 ** -24)[~inf].all()), f"{what}: lse"


def draw_sinks(rng, heads):
    if rng.random() < 0.5:
        return None
    s = torch.randn(heads, device=DEV)
    for _ in range(2):
        s[rng.randrange(heads)] = rng.choice([math.inf, -math.inf, 0.0, 50.0])
    return s


def results(q8, call, kind):
    """fp32 results of a call, whose other output types and second run agree with them bit for bit."""
    o, lse = call(q8.Q8_TYPE_F32)
    assert torch.equal(o, call(q8.Q8_TYPE_F32)[0]) and torch.equal(call(None)[0], o.to(DT[kind]))
    n = o.shape[0]
    assert torch.equal(call(q8.Q8_TYPE_Q8_0)[0].view(n, -1), q8.quantize_act(o.view(n, -1)))
    assert q8.q8_last_error() == 0
    return o.double(), lse.double()


@pytest.mark.parametrize("seed", range(80))
def test_decode_draws(q8, seed):
    rng = random.Random(seed)
    torch.manual_seed(seed)
    kind, dim, kv = rng.choice(["bf16", "f16", "q8"]), rng.choice([64, 128, 256, 512]), rng.choice([1, 1, 2, 3, 5])
    group, page = rng.choice([1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 24, 33, 64]), rng.choice([16, 32, 64, 128, 256])
    seqs, top = rng.choice([1, 1, 2, 3, 7, 31, 32, 33, 64, 150]), rng.choice([1, 17, 70, 300, 1000, 5000])
    while seqs * top * kv * dim > 20_000_000 and top > 1:
        top //= 2
    lens = [rng.choice([0, 1, top, rng.randint(0, top), rng.randint(0, top)]) for _ in range(seqs)]
    window = rng.choice([0, 0, 0, 1, rng.randint(1, top + 5), (1 << 32) - 1])
    qtype = rng.choice(["bf16", "f16"]) if kind == "q8" else kind
    heads, layers = kv * group, rng.choice([1, 2])
    layer, scale = rng.randrange(layers), rng.choice([dim ** -0.5, 0.05])
    code = {"q8": q8.Q8_TYPE_Q8_0, "f16": q8.Q8_TYPE_F16, "bf16": q8.Q8_TYPE_BF16}[kind]
    need = [-(-n // page) for n in lens]
    table = torch.full((seqs, max(need) + rng.choice([1, 9])), -7, dtype=torch.int32)
    n_pages, order = sum(need) + 2, torch.randperm(sum(need) + 2).int()
    unseen, at = torch.ones(n_pages, page, dtype=torch.bool), 0
    for i, n in enumerate(lens):
        table[i, :need[i]] = order[at:at + need[i]]
        at += need[i]
        rows = torch.arange(max(0, n - window) if window else 0, n)
        unseen[table[i, rows // page].long(), rows % page] = False
    unseen = unseen.to(DEV)[None, :, None, :, None]
    values, pools = [], []
    for _ in range(2):
        if kind == "q8":
            quants = torch.randint(-127, 128, (layers, n_pages, kv, page, dim), dtype=torch.int8, device=DEV)
            d = (torch.rand(layers, n_pages, kv, page, dim // 32, device=DEV) * rng.choice([1e-3, 1.0, 30.0]) / 64).half()
            values.append((quants.double() * d.double().repeat_interleave(32, -1))[layer])
            d = torch.where(unseen, torch.full_like(d, math.nan), d)
            pools.append(torch.cat([quants.view(torch.uint8).flatten(3), d.contiguous().view(torch.uint8).flatten(3)], -1).flatten(2))
        else:
            x = torch.randn(layers, n_pages, kv, page, dim, device=DEV).to(DT[kind])
            values.append(x.double()[layer])
            pools.append(torch.where(unseen, torch.full_like(x, rng.choice([math.nan, math.inf])), x))
    cache = q8.KVCache(*pools, code, page, kv, dim)
    q = torch.randn(seqs, heads + 2, dim, device=DEV).to(DT[qtype])[:, 1:1 + heads]
    sinks, t = draw_sinks(rng, heads), table.to(DEV)
    n_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = results(q8, lambda o: q8.attn_decode(q, cache, layer, t, n_t, scale=scale, window=window, sinks=sinks, out_type=o,
                                                    want_lse=True), qtype)
    for i in {0, seqs - 1, *(rng.randrange(seqs) for _ in range(8))}:
        n = lens[i]
        k, v = (x[table[i, :need[i]].long().to(DEV)].transpose(0, 1).reshape(kv, -1, dim)[:, :n].repeat_interleave(group, 0) for x in values)
        see = torch.ones(1, n, dtype=torch.bool, device=DEV)
        see[:, :max(0, n - window) if window else 0] = False
        compare(out[i][:, None], lse[i][:, None], q[i].double()[:, None], k, torch.where(see[0][:, None], v, 0.0), see, scale,
                None if sinks is None else sinks.double(), "bf16" if kind == "bf16" else "f16", f"sequence {i} of {n}")


@pytest.mark.parametrize("seed", range(80))
def test_prompt_draws(q8, seed):
    rng = random.Random(1000 + seed)
    torch.manual_seed(seed)
    kind, dim, kv = rng.choice(["bf16", "f16"]), rng.choice([64, 128, 256, 512]), rng.choice([1, 1, 2, 3])
    group, seqs = rng.choice([1, 2, 3, 5, 7, 8, 12, 16, 24, 64, 130]), rng.choice([1, 1, 2, 5, 20, 33, 100, 400])
    heads, top = kv * group, rng.choice([1, 5, 64, 129, 300, 700, 2000])
    while seqs * top * heads * dim > 30_000_000 and top > 1:
        top //= 2
    queries = [rng.choice([0, 1, top, rng.randint(0, top), rng.randint(0, top)]) for _ in range(seqs)]
    queries[0] = max(1, queries[0])
    keys = [max(0, n + rng.choice([0, 0, 0, rng.randint(-50, 200), rng.randint(0, 900), -n])) for n in queries]
    window, scale = rng.choice([0, 0, 1, rng.randint(1, 400), (1 << 32) - 1]), rng.choice([dim ** -0.5, 0.05])
    q0, k0 = ([0, *torch.tensor(x).cumsum(0).tolist()] for x in (queries, keys))
    q = torch.randn(q0[-1], heads + 1, dim, device=DEV).to(DT[kind])[:, :heads]
    both = torch.randn(k0[-1] + rng.choice([0, 150]), 2 * kv + 1, dim, device=DEV).to(DT[kind])
    both[k0[-1]:] = math.nan
    k, v = both[:, :kv], both[:, kv:2 * kv]
    sinks = draw_sinks(rng, heads)
    qs, ks = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (q0, k0))
    out, lse = results(q8, lambda o: q8.attn_prompt(q, k, v, qs, ks, scale=scale, window=window, sinks=sinks, out_type=o, want_lse=True), kind)
    for i in {0, seqs - 1, *(rng.randrange(seqs) for _ in range(4))}:
        a, b = slice(q0[i], q0[i + 1]), slice(k0[i], k0[i + 1])
        if queries[i] == 0:
            continue
        last, j = torch.arange(queries[i], device=DEV)[:, None] + keys[i] - queries[i], torch.arange(keys[i], device=DEV)
        see = (j <= last) & ((j > last - window) if window else True)
        hs = sorted({rng.randrange(heads) for _ in range(4)})
        part = lambda x, s, h: x[s][:, h].double().transpose(0, 1)
        compare(out[a][:, hs].transpose(0, 1), lse[a][:, hs].transpose(0, 1), part(q, a, hs), part(k, b, [h // group for h in hs]),
                part(v, b, [h // group for h in hs]), see, scale, None if sinks is None else sinks[hs].double(), kind,
                f"sequence {i} ({queries[i]}, {keys[i]})")
