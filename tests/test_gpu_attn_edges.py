"""GPU tests of the attention kernels at the ends of their numbers."""
import numpy as np
import pytest

from tests.attn_plain import attend
from tests.test_gpu_attn import check_prompt

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"


@pytest.fixture(scope="module")
def q8():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_quantized_matmul_gb300 import build
    build.build()
    import q8_quantized_matmul_gb300 as m
    torch.cuda.set_device(0)
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def far_below(n, dim, seed):
    """Keys and values [n, 1, dim] fp16: every 128th key is 17.5 ahead of the others in natural logarithms and has
    values of zero, the others have values of 500 to 1000: the output is what the small weights add up to."""
    g = torch.Generator().manual_seed(seed)
    k = torch.full((n, 1, dim), -17.5 * dim ** -0.5)
    v = torch.rand((n, 1, dim), generator=g) * 500 + 500
    k[5::128], v[5::128] = 0.0, 0.0
    return k.half().to(DEV), v.half().to(DEV)


def check_far_below(got, k, v, rows, last, dim, what):
    """The bound of tests/attn_plain.py with weights of 8 bits (2^-8 of the weighted mean; fp16 keeps at least 6 of a
    weight at 2^-25 of the largest: the rest) plus half a step of fp16 below its normal numbers, 2^-25, counted in units
    2^7 below the largest weight: 2^-32 |v| a key."""
    kf, vf = k.cpu().double().numpy()[:, 0], v.cpu().double().numpy()[:, 0]
    q = np.ones((1, dim))
    for r in rows:
        n = last(r) + 1
        ref, lse, bound, _ = attend(q, kf[:n], vf[:n], np.ones((1, n), bool), dim ** -0.5, None, "bf16", "f32")
        bound = bound + 2.0 ** -32 * np.abs(vf[:n]).sum(0) / np.exp(lse[0] - (kf[:n] @ q[0] * dim ** -0.5).max())
        assert np.all(ref[0] > 2.0 * bound[0])                       # a kernel that loses these weights cannot pass
        err = np.abs(got[r] - ref)
        assert np.all(err <= bound), f"{what}, row {r}: {(err / bound).max():.2f} of the bound"


@pytest.mark.parametrize("dim,heads", [(64, 2), (128, 12), (256, 2), (512, 2), (256, 24), (512, 24)])
def test_decode_sums_weights_far_below_the_largest(q8, dim, heads):
    lens, page = [3000, 700], 64
    cache = q8.KVCache.empty(q8.Q8_TYPE_F16, 1, 60, page, 1, dim)
    table = i32([list(range(47)), [*range(47, 58), *[-1] * 36]])
    rows = [far_below(n, dim, i) for i, n in enumerate(lens)]
    for i, (k, v) in enumerate(rows):
        pos = torch.arange(lens[i], dtype=torch.int32, device=DEV)
        q8.kv_append(cache, 0, None, k.float(), v.float(), pos, torch.full_like(pos, i), table)
    q = torch.ones(2, heads, dim, device=DEV, dtype=torch.float16)
    got = q8.attn_decode(q, cache, 0, table, i32(lens), out_type=q8.Q8_TYPE_F32).cpu().double().numpy()
    assert q8.q8_last_error() == 0
    for i, (k, v) in enumerate(rows):
        for h in (0, heads - 1):
            check_far_below(got[i, h][None], k, v, [0], lambda r: lens[i] - 1, dim, f"sequence {i} head {h}")


@pytest.mark.parametrize("dim", [64, 128, 256, 512])
def test_prompt_sums_weights_far_below_the_largest(q8, dim):
    n = 700
    k, v = far_below(n, dim, dim)
    q = torch.ones(n, 2, dim, device=DEV, dtype=torch.float16)
    got = q8.attn_prompt(q, k, v, i32([0, n]), out_type=q8.Q8_TYPE_F32).cpu().double().numpy()
    assert q8.q8_last_error() == 0
    for h in range(2):
        check_far_below(got[:, h], k, v, [0, 4, 5, 6, 127, 128, 300, 699], lambda r: r, dim, f"head {h}")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim,heads", [(64, 2), (128, 2), (512, 24)])
def test_very_large_scores(q8, kind, dim, heads):
    """Scores of 2^23 to 2^25 (log2 units, steps of 1 to 4): equal keys share the weight, whatever the distance of their scores' roundings."""
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    n = 150
    q = torch.full((n, heads, dim), 1000.0, device=DEV).to(dt)
    k = torch.full((n, 1, dim), 1000.0, device=DEV).to(dt)
    v = torch.full((n, 1, dim), 3.0, device=DEV).to(dt)
    o = q8.attn_prompt(q, k, v, i32([0, n]), out_type=q8.Q8_TYPE_F32)
    cache = q8.KVCache.empty(q8.Q8_TYPE_F16 if kind == "f16" else q8.Q8_TYPE_BF16, 1, 5, 32, 1, dim)
    pos, table = torch.arange(n, dtype=torch.int32, device=DEV), i32([[0, 1, 2, 3, 4]])
    q8.kv_append(cache, 0, None, k.float(), v.float(), pos, torch.zeros_like(pos), table)
    d = q8.attn_decode(q[:1].contiguous(), cache, 0, table, i32([n]), out_type=q8.Q8_TYPE_F32)
    assert q8.q8_last_error() == 0
    u = 2.0 ** (-11 if kind == "f16" else -8)                       # a weight's rounding, and the sums'
    for x in (o, d):
        assert (x - 3.0).abs().max() <= 3.0 * (u + 2.0 ** -18)


@pytest.mark.parametrize("dim,heads", [(64, 4), (128, 4), (256, 4), (512, 20)])
def test_infinite_sinks(q8, dim, heads):
    """exp(sink) = 0 adds nothing; exp(sink) = inf leaves nothing for the keys: zeros, and a denominator of inf."""
    n = 200
    g = torch.Generator().manual_seed(dim)
    q, k, v = (torch.randn((n, h, dim), generator=g).half().to(DEV) for h in (heads, 1, 1))
    sinks = torch.zeros(heads, device=DEV)
    sinks[1], sinks[2] = -float("inf"), float("inf")
    cache = q8.KVCache.empty(q8.Q8_TYPE_F16, 1, 8, 32, 1, dim)
    pos, table = torch.arange(n, dtype=torch.int32, device=DEV), i32([list(range(8))])
    q8.kv_append(cache, 0, None, k.float(), v.float(), pos, torch.zeros_like(pos), table)
    prompt = lambda s: q8.attn_prompt(q, k, v, i32([0, n]), sinks=s, want_lse=True)
    decode = lambda s: q8.attn_decode(q[-2:].contiguous(), cache, 0, table.repeat(2, 1), i32([n, 0]), sinks=s, want_lse=True)
    for call in (prompt, decode):
        o, lse = call(sinks)
        plain, plain_lse = call(None)
        zero, zero_lse = call(torch.zeros_like(sinks))
        assert torch.equal(o[:, 1], plain[:, 1]) and torch.equal(lse[:, 1], plain_lse[:, 1])
        assert torch.all(o[:, 2] == 0) and torch.all(lse[:, 2] == float("inf"))
        rest = [h for h in range(heads) if h not in (1, 2)]
        assert torch.equal(o[:, rest], zero[:, rest]) and torch.equal(lse[:, rest], zero_lse[:, rest])
    assert q8.q8_last_error() == 0


@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_infinite_values_beside_sequences_without_keys(q8, dim):
    """Sequences of one key, each with an infinity among its values, among many that have queries and no key, beside one
    of 131 000 keys, with which sequences of no key and of one lie together in the list of tiles: each row of one key is
    that key's values."""
    rng = np.random.default_rng(dim)
    one = rng.random(200_000) < 0.1
    qlen, klen = np.where(one, 1, 2), np.where(one, 1, 0)
    qlen[77], klen[77] = 1, 131_000
    q0, k0 = (np.concatenate([[0], np.cumsum(x)]) for x in (qlen, klen))
    one[77] = False
    q = torch.randn(int(q0[-1]), 1, dim, device=DEV).half()
    k, v = (torch.randn(int(k0[-1]), 1, dim, device=DEV).half() for _ in range(2))
    keys = torch.from_numpy(k0[:-1][one]).to(DEV)
    rows = torch.from_numpy(q0[:-1][one]).to(DEV)
    v[keys, 0, keys % dim] = float("inf")
    for _ in range(3):
        o = q8.attn_prompt(q, k, v, i32(q0), i32(k0))
        assert torch.equal(o[rows], v[keys])
        none = torch.ones(q.shape[0], dtype=torch.bool, device=DEV)
        none[rows] = none[int(q0[77])] = False
        assert torch.all(o[none] == 0) and torch.isfinite(o[int(q0[77])]).all()
    assert q8.q8_last_error() == 0


@pytest.mark.parametrize("tokens,seqs", [(3000, 400), (1 << 21, 1 << 20)])
def test_prompt_starts_that_fall(q8, tokens, seqs):
    """Starts that go back and forth make each second sequence all the rows, 2^32 tiles in the larger case: an error,
    soon, nothing outside the outputs, and the next call is right."""
    q = torch.randn(tokens, 2, 64, device=DEV).half()
    k = torch.randn(tokens, 1, 64, device=DEV).half()
    n = tokens // 100
    small = i32([0, n // 3, n])
    ref = q8.attn_prompt(q[:n], k, k, small)
    start = torch.zeros(seqs + 1, dtype=torch.int32, device=DEV)
    start[1::2] = tokens
    for _ in range(2):
        q8.attn_prompt(q, k, k, start)
        assert q8.q8_last_error() == q8.Q8_ERANGE
    assert torch.equal(q8.attn_prompt(q[:n], k, k, small), ref)
    assert q8.q8_last_error() == 0


@pytest.mark.parametrize("dim,heads,seqs", [(512, 64, 3), (256, 24, 3), (512, 24, 120), (256, 64, 40), (512, 64, 160)])
def test_decode_kernels_agree_on_either_side_of_their_rule(q8, dim, heads, seqs):
    """The same sequences with rows of pages that leave room for few positions and for many, which run on different
    kernels: each within half a step of bf16 of the weighted mean of |v| (below 4) for its weights, and the logarithm of
    the denominator within 2 (D + 8) 2^-23 of sum |q k| scale (below 16 for 512 normal values) for the scores' sums."""
    page, n_pages = 16, 8 * seqs
    g = torch.Generator().manual_seed(seqs)
    cache = q8.KVCache.empty(q8.Q8_TYPE_BF16, 1, n_pages, page, 1, dim)
    for pool in (cache.k, cache.v):
        pool.view(torch.bfloat16).copy_(torch.randn(pool.view(torch.bfloat16).shape, generator=g).clamp(-4, 4))
    lens = torch.randint(0, 65, (seqs,), generator=g).int()
    lens[0], lens[-1] = 0, 64
    table = torch.randperm(n_pages, generator=g)[:4 * seqs].view(seqs, 4).int().to(DEV)
    wide = torch.full((seqs, 40), -1, dtype=torch.int32, device=DEV)
    wide[:, :4] = table
    q = torch.randn(seqs, heads, dim, generator=g).bfloat16().to(DEV)
    for window in (0, 10):
        (a, la), (b, lb) = (q8.attn_decode(q, cache, 0, t, lens.to(DEV), window=window, out_type=q8.Q8_TYPE_F32, want_lse=True)
                            for t in (table, wide))
        assert (a - b).abs().max() <= 2 * 4 * (2.0 ** -8 + 2.0 ** -18)
        assert torch.equal(la.isinf(), lb.isinf()) and (la - lb)[~la.isinf()].abs().max() <= 2 * 2 * 520 * 16 * 2.0 ** -23
    assert q8.q8_last_error() == 0


@pytest.mark.parametrize("window", [1, 64, 129, 300])
@pytest.mark.parametrize("heads,kv", [(2, 1), (20, 1), (6, 3)])
def test_prompt_windows_of_heads_of_512(q8, window, heads, kv):
    check_prompt(q8, "bf16", [300, 5, 0, 140], [300, 205, 30, 90], heads=heads, kv=kv, dim=512, window=window, sinks=True, seed=window)


def test_raw_calls_agree_with_the_tensor_helpers(q8):
    """The package's bindings of the C entry points, one per call, against the helpers on the same tensors."""
    n, heads, kv, dim, page, pages = 100, 4, 2, 64, 16, 20
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((n, h, dim), generator=g).to(DEV) for h in (heads, kv, kv))
    cs = torch.randn((n, dim), generator=g).to(DEV)
    pos, seq = torch.arange(n, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
    row, other, many = i32([0]), i32([1]), i32([n])
    state = []
    for raw in (False, True):
        c = q8.KVCache.empty(q8.Q8_TYPE_Q8_0, 1, pages, page, kv, dim)
        table, lens, refs = torch.full((2, 9), -1, dtype=torch.int32, device=DEV), i32([0, 0]), i32([1] + [0] * (pages - 1))
        if not raw:
            q8.kv_reserve(c, table, lens, refs, row, many)
            q16, k16, v16 = q8.kv_append(c, 0, q, k, v, pos, seq, table, cs, 1, torch.float16, want_kv=True)
            q8.kv_fork(c, table, lens, refs, row, other)
            o, lse = q8.attn_decode(q16[-2:].contiguous(), c, 0, table, lens, window=50, want_lse=True)
            p, plse = q8.attn_prompt(q16, k16, v16, i32([0, 40, n]), want_lse=True)
            q8.kv_free(c, table, lens, refs, row)
            t2, r2, used = q8.kv_compact(c, table, lens, refs)
            q8.kv_copy(c, row, i32([pages - 1]))
        else:
            s, f16, sc = c.struct, q8.Q8_TYPE_F16, dim ** -0.5
            new = lambda t: torch.empty_like(t)
            assert q8.q8_kv_reserve(s, table, 9, 9, 2, lens, refs, row, many, 1) == 0
            q16, k16, v16 = q.half(), k.half(), v.half()
            assert q8.q8_kv_append(q16, k16, v16, f16, s, 0, q, heads * dim, k, kv * dim, v, kv * dim, heads, kv, dim, pos, seq, table,
                                   9, 9, 2, cs, n, dim, 1, n) == 0
            assert q8.q8_kv_fork(s, table, 9, 9, 2, lens, refs, row, other, 1) == 0
            o, lse = new(q16[-2:]), torch.empty(2, heads, device=DEV)
            assert q8.q8_attn_decode(o, f16, lse, q16[-2:].contiguous(), heads * dim, f16, s, 0, table, 9, 9, lens, 2, heads, sc, 50, None) == 0
            p, plse = new(q16), torch.empty(n, heads, device=DEV)
            start = i32([0, 40, n])
            assert q8.q8_attn_prompt(p, f16, plse, q16, k16, v16, f16, heads * dim, kv * dim, kv * dim, start, None, 2, n, n, heads, kv,
                                     dim, sc, 0, None) == 0
            assert q8.q8_kv_free(s, table, 9, 9, 2, lens, refs, row, 1) == 0
            t2, r2, used = new(table), new(refs), torch.empty((), dtype=torch.int32, device=DEV)
            assert q8.q8_kv_compact(s, t2, table, 9, 9, 2, r2, refs, used) == 0
            last = i32([pages - 1])
            assert q8.q8_kv_copy(s, row, last, 1) == 0
        assert q8.q8_last_error() == 0
        state.append([q16, k16, v16, o, lse, p, plse, t2, r2, used, table, lens, refs, c.k, c.v])
    for a, b in zip(*state):
        assert torch.equal(a, b)


@pytest.mark.parametrize("out", [None, "f32", "q8"])
@pytest.mark.parametrize("kind,dim,heads,kv,lens", [
    ("bf16", 512, 64, 2, [1, 125, 40, 0, 300, 7, 90, 128, 129] * 16),     # 256 units with a step or more over 152 CTAs
    ("f16", 256, 33, 5, [1, 70, 20, 0] * 40),                             # 600 of one step: several a CTA
    ("bf16", 256, 17, 1, [4000] * 3 + [9] * 300)])                        # long ones that are cut beside short ones
def test_decode_several_units_of_wide_heads_in_a_cta(q8, kind, dim, heads, kv, lens, out):
    """More (sequence, key-value head, 64 query heads) than CTAs, and shares that hold many short ones: every row against
    the definition in 64 bits on the GPU, with the error terms of tests/attn_plain.py."""
    page, dt = 64, torch.bfloat16 if kind == "bf16" else torch.float16
    n, group, need = len(lens), heads, [-(-m // 64) for m in lens]
    heads *= kv
    g = torch.Generator(device=DEV).manual_seed(dim)
    normal = lambda *s: torch.randn(s, generator=g, device=DEV).to(dt)
    k, v = normal(1, sum(need), kv, page, dim), normal(1, sum(need), kv, page, dim)
    table, at = np.full((n, 64), -1, np.int32), 0
    order = np.random.default_rng(dim).permutation(sum(need))
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    cache = q8.KVCache(k, v, q8.Q8_TYPE_BF16 if kind == "bf16" else q8.Q8_TYPE_F16, page, kv, dim)
    q, sinks = normal(n, heads, dim), torch.randn(heads, generator=g, device=DEV)
    code = {None: None, "f32": q8.Q8_TYPE_F32, "q8": q8.Q8_TYPE_Q8_0}[out]
    call = lambda c: q8.attn_decode(q, cache, 0, torch.from_numpy(table).to(DEV), i32(lens), sinks=sinks, out_type=c, want_lse=True)
    o, lse = call(code)
    assert q8.q8_last_error() == 0
    if out == "q8":
        o32, _ = call(q8.Q8_TYPE_F32)
        assert torch.equal(o.view(n, -1), q8.quantize_act(o32.view(n, -1)))
        return
    half = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[kind]
    scale = dim ** -0.5
    for i, m in enumerate(lens):
        pages = torch.from_numpy(table[i, :need[i]]).long().to(DEV)
        kk, vv = (x[0, pages].transpose(0, 1).reshape(kv, -1, dim)[:, :m].double().repeat_interleave(group, 0) for x in (k, v))
        qq = q[i].double()[:, None]
        z = (qq @ kk.transpose(1, 2))[:, 0] * scale
        full = torch.logsumexp(torch.cat([z, sinks.double()[:, None]], 1), 1)
        w = torch.exp(z - full[:, None])
        ref, mean = (w[:, None] @ vv)[:, 0], (w[:, None] @ vv.abs())[:, 0]
        dz = ((dim + 8) * 2.0 ** -23 * scale * (qq.abs() @ kk.abs().transpose(1, 2))[:, 0] + 4 * z.abs() * 2.0 ** -23).amax(1) if m else torch.zeros_like(full)
        sums = 2.0 ** -21 + (m / 8 + 16) * 2.0 ** -23
        bound = mean * (half + 2 * dz[:, None] + sums) + (2.0 ** -24 if out else half) * ref.abs() + 1e-30
        if kind == "f16" and m:
            bound = bound + 2.0 ** -32 * m * vv.abs().amax(1)
        if kind == "f16" and not out:
            bound = bound + 2.0 ** -25                                # half a step of fp16 below its normal numbers
        err = (o[i].double() - ref).abs()
        assert torch.all(err <= bound), f"sequence {i} of {m}: {float((err / bound).max()):.2f} of the bound"
        assert torch.all((lse[i].double() - full).abs() <= 2 * dz + sums + 8 * full.abs() * 2.0 ** -24), f"lse of sequence {i}"
    assert torch.equal(o, call(code)[0])
