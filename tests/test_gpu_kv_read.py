"""GPU tests of q8_kv_read: the rows that a plain look-up of the pages gives, bit for bit."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


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
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def code(q8, name):
    return {"f32": q8.Q8_TYPE_F32, "f16": q8.Q8_TYPE_F16, "bf16": q8.Q8_TYPE_BF16, "q8": q8.Q8_TYPE_Q8_0}[name]


def filled(q8, kind, layers, pages, page, kv, dim, seed=0):
    """A cache of random values, and its values [layers, pages, kv, page, dim] for K and V in fp32."""
    rng = np.random.default_rng(seed)
    cache = q8.KVCache.empty(code(q8, kind), layers, pages, page, kv, dim)
    values = []
    for pool in (cache.k, cache.v):
        if kind == "q8":
            q = rng.integers(-127, 128, (layers, pages, kv, page, dim // 32, 32)).astype(np.int8)
            d = rng.uniform(1e-3, 1e-1, (layers, pages, kv, page, dim // 32)).astype(np.float16)
            raw = np.concatenate([q.reshape(layers, pages, kv, -1).view(np.uint8), d.reshape(layers, pages, kv, -1).view(np.uint8)], -1)
            values.append((q * d[..., None].astype(np.float32)).reshape(layers, pages, kv, page, dim))
        else:
            x = torch.from_numpy(rng.standard_normal((layers, pages, kv, page, dim)).astype(np.float32)).to(DT[kind])
            raw = x.view(torch.uint8).numpy()
            values.append(x.float().numpy())
        pool.copy_(torch.from_numpy(raw.reshape(layers, pages, -1)))
    return cache, values


def rows_of(values, layer, table, page, spans):
    """spans: (row, first, count) of each sequence -> [rows, kv, dim]."""
    out = [np.zeros((0,) + values.shape[2:3] + values.shape[4:], np.float32)]
    for r, first, count in spans:
        for t in range(first, first + count):
            out.append(values[layer, table[r][t // page], :, t % page][None])
    return np.concatenate(out)


@pytest.mark.parametrize("kind,out", [("q8", "bf16"), ("q8", "f16"), ("q8", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f16", "f32"), ("bf16", "f16"),
                                      ("f16", "bf16")])
@pytest.mark.parametrize("kv,dim,page", [(1, 64, 16), (3, 128, 32), (2, 256, 128), (1, 512, 256), (8, 64, 64)])
def test_rows(q8, kind, out, kv, dim, page):
    rng = np.random.default_rng(kv + dim)
    cache, (k, v) = filled(q8, kind, 2, 12, page, kv, dim)
    table = rng.permutation(12).reshape(3, 4).astype(np.int32)
    spans = [(2, page - 1, 2), (0, 0, 0), (0, 3, 3 * page), (1, 0, 1), (2, 2 * page, 2 * page)]
    start = np.concatenate([[0], np.cumsum([c for _, _, c in spans])])
    n = int(start[-1])
    got = q8.kv_read(cache, 1, i32(table), i32(start), n, first=i32([f for _, f, _ in spans]), seqs=i32([r for r, _, _ in spans]),
                     out_type=code(q8, out))
    assert q8.q8_last_error() == 0
    for g, x in zip(got, (k, v)):
        want = torch.from_numpy(rows_of(x, 1, table, page, spans)).to(DT[out])
        assert g.dtype == DT[out] and torch.equal(g.cpu(), want)


def test_whole_rows_by_default_and_into_a_wider_tensor(q8):
    cache, (k, v) = filled(q8, "q8", 1, 8, 16, 2, 64)
    table = np.array([[3, 1, -1], [7, 0, 2]], np.int32)
    spans = [(0, 0, 20), (1, 0, 33)]
    want = [torch.from_numpy(rows_of(x, 0, table, 16, spans)).bfloat16() for x in (k, v)]
    got = q8.kv_read(cache, 0, i32(table), i32([0, 20, 53]), 53)
    assert all(torch.equal(g.cpu(), w) for g, w in zip(got, want))
    both = torch.full((60, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    q8.kv_read(cache, 0, i32(table), i32([0, 20, 53]), 55, out=(both[:, :2], both[:, 2:]))
    assert torch.equal(both[:53].cpu(), torch.cat(want, 1)) and (both[53:] == 7).all()       # rows of no sequence stay


def test_bad_pages_rows_and_starts(q8):
    cache, (k, _) = filled(q8, "f16", 1, 4, 16, 1, 64)

    def call(table, start, n, **kw):
        k_out = torch.full((n, 1, 64), 7.0, dtype=torch.float16, device=DEV)
        q8.kv_read(cache, 0, i32(table), i32(start), n, out=(k_out, torch.empty_like(k_out)), **kw)
        return k_out.cpu()[:, 0], q8.q8_last_error()

    for page in (-1, 4, 2 ** 31 - 1, -2 ** 31):                       # no such page: zeros
        got, rc = call([[0, page]], [0, 20], 20)
        assert rc == q8.Q8_ERANGE and torch.equal(got[:16].float(), torch.from_numpy(k[0, 0, 0])) and not got[16:].any()
    for first in (-1, 13, 2 ** 31 - 1, -2 ** 31):                     # positions outside the row's pages
        got, rc = call([[2, 3]], [0, 20], 20, first=i32([first]))
        inside = [i for i in range(20) if 0 <= first + i < 32]
        assert rc == q8.Q8_ERANGE and not got[[i for i in range(20) if i not in inside]].any()
        for i in inside:
            assert torch.equal(got[i].float(), torch.from_numpy(k[0, 2 + (first + i) // 16, 0, (first + i) % 16]))
    for row in (-1, 1, 2 ** 31 - 1):
        got, rc = call([[2, 3]], [0, 5], 5, seqs=i32([row]))
        assert rc == q8.Q8_ERANGE and not got.any()
    got, rc = call([[2, 3]], [0, 9], 5)                               # beyond n_k: cut
    assert rc == q8.Q8_ERANGE and torch.equal(got.float(), torch.from_numpy(k[0, 2, 0, :5]))
    got, rc = call([[2, 3], [0, 1], [1, 0]], [0, 4, 2, 5], 5)         # starts that fall: an error, nothing outside touched
    assert rc == q8.Q8_ERANGE
    got, rc = call([[2, 3]], [2, 5], 5)                               # does not start at 0
    assert rc == q8.Q8_ERANGE and (got[:2] == 7).all() and torch.equal(got[2:].float(), torch.from_numpy(k[0, 2, 0, :3]))
    got, rc = call([[2, 3]], [-4, 5], 5)                              # below 0: cut
    assert rc == q8.Q8_ERANGE and torch.equal(got.float(), torch.from_numpy(k[0, 2, 0, :5]))
    assert call([[2, 3]], [0, 5], 5)[1] == 0


def test_far_positions_and_many_sequences(q8):
    """2000 sequences of one token, far apart in rows of 4000 pages."""
    cache, (k, v) = filled(q8, "bf16", 1, 64, 16, 1, 64)
    rng = np.random.default_rng(1)
    n = 2000
    table = rng.integers(0, 64, (n, 4000)).astype(np.int32)
    first = rng.integers(0, 64000, n)
    got = q8.kv_read(cache, 0, i32(table), i32(np.arange(n + 1)), n, first=i32(first))
    at = table[np.arange(n), first // 16]
    for g, x in zip(got, (k, v)):
        assert np.array_equal(g.float().cpu().numpy()[:, 0], x[0, at, 0, first % 16])
    assert q8.q8_last_error() == 0


def test_pools_and_rows_beyond_32_bits(q8):
    page, kv, dim, pages = 256, 1, 256, 40000                         # 5.2 GB a pool
    cache = q8.KVCache.empty(q8.Q8_TYPE_BF16, 1, pages, page, kv, dim)
    table = [[39999, 0, 35000]]
    want = torch.randn(3 * page, kv, dim, device=DEV).bfloat16()
    for i, p in enumerate(table[0]):
        cache.k[0, p].copy_(want[i * page:(i + 1) * page].view(-1).view(torch.uint8))
    n, stride = 3 * page - 100, 1 << 22
    rows = torch.empty(n * stride, dtype=torch.bfloat16, device=DEV).view(n, stride)[:, :dim].unsqueeze(1)
    v = torch.empty(n, kv, dim, dtype=torch.bfloat16, device=DEV)
    q8.kv_read(cache, 0, i32(table), i32([0, n]), n, first=i32([100]), out=(rows, v))
    assert torch.equal(rows, want[100:]) and not v.any() and q8.q8_last_error() == 0


@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_prompt_in_parts(q8, kind):
    """A prompt attended in two parts, the second over what kv_read gives, has the whole prompt's rows: with a 16-bit
    cache to the bit, with Q8_0 as over the cache's own values."""
    n, cut, heads, kv, dim, page = 300, 170, 4, 2, 128, 32
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = (torch.randn(n, h, dim, generator=g, device=DEV) for h in (heads, kv, kv))
    cache = q8.KVCache.empty(code(q8, kind), 1, 10, page, kv, dim)
    table, pos = i32([np.random.default_rng(0).permutation(10)]), i32(np.arange(n))
    zero = torch.zeros_like(pos)
    qs, ks, vs = q8.kv_append(cache, 0, q, k, v, pos, zero, table, dtype=torch.bfloat16, want_kv=True)
    kr, vr = q8.kv_read(cache, 0, table, i32([0, n]), n)
    if kind == "bf16":
        assert torch.equal(kr, ks) and torch.equal(vr, vs)
    whole = q8.attn_prompt(qs, kr, vr, i32([0, n]))
    k1, v1 = q8.kv_read(cache, 0, table, i32([0, cut]), cut)
    part1 = q8.attn_prompt(qs[:cut], k1, v1, i32([0, cut]))
    part2 = q8.attn_prompt(qs[cut:].contiguous(), kr, vr, i32([0, n - cut]), i32([0, n]))
    both = torch.cat([part1, part2])
    # the tiles of keys are the same, a row's place in its tile of queries is not: 2^-7 of the largest value covers the
    # 16-bit weights' rounding against another running maximum
    assert (both.float() - whole.float()).abs().max() <= 2.0 ** -7 * vr.float().abs().max()


def test_captured_and_refused(q8):
    cache, _ = filled(q8, "q8", 1, 4, 16, 2, 64)
    table, start = i32([[1, 3]]), i32([0, 30])
    want = q8.kv_read(cache, 0, table, start, 30)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = q8.kv_read(cache, 0, table, start, 30)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for bad in (lambda: q8.kv_read(cache, 1, table, start, 30), lambda: q8.kv_read(cache, 0, table, i32([0, 1, 2]), 2),
                lambda: q8.kv_read(cache, 0, table, start, 30, first=i32([0, 0])), lambda: q8.kv_read(cache, 0, table, start.long(), 30),
                lambda: q8.kv_read(cache, 0, table, start, 30, out_type=8), lambda: q8.kv_read(cache, 0, table.cpu(), start, 30),
                lambda: q8.kv_read(cache, 0, table, start, 30, out=(want[0][:20], want[1][:20])),
                lambda: q8.kv_read(cache, 0, table, start, 30, out=(want[0], None))):
        with pytest.raises((TypeError, ValueError, q8.Q8Error)):
            bad()
    assert q8.kv_read(cache, 0, table, i32([0, 0]), 0)[0].shape == (0, 2, 64)
