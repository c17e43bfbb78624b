"""GPU parity of the paged key-value cache's attention (q8_attn_decode, q8_attn_prompt) against its definition in
64 bits; the tolerances are derived in tests/attn_plain.py."""
import numpy as np
import pytest

from tests.attn_plain import attend

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


DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def f64(t):
    return t.detach().cpu().double().numpy()


def dequantise(rows, dim):
    """Quantised rows as fp64: the quantiser of the library's activations, on the host."""
    x = rows.reshape(-1, dim // 32, 32).astype(np.float32)
    d = np.abs(x).max(-1) / np.float32(127)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(d[..., None] > 0, x / d[..., None], 0)
    q = np.trunc(y) + np.where(np.abs(y - np.trunc(y)) >= 0.5, np.sign(y), 0)
    d16 = d.astype(np.float16)
    return q.astype(np.int8).reshape(rows.shape), d16.reshape(*rows.shape[:-1], dim // 32)


class Pool:
    """A cache filled from fp32 rows; everything that holds no position of a sequence is poisoned."""

    def __init__(self, q8, kind, lens, kv, dim, page, seed, v_scale=1.0, strided=False, layers=1, layer=0):
        rng = np.random.default_rng(seed)
        self.lens, self.kind = lens, kind
        need = [-(-n // page) for n in lens]
        n_pages, width = sum(need) + 2, max(max(need), 1) + 1
        order = rng.permutation(n_pages)
        table = np.full((len(lens), width), 1 << 28, np.int32)       # never looked up beyond the sequence
        at = 0
        for i, k in enumerate(need):
            table[i, :k] = order[at:at + k]
            at += k
        self.rows = []                                               # exact values, [seq][k / v] [len, kv, dim]
        code = {"q8": q8.Q8_TYPE_Q8_0, "f16": q8.Q8_TYPE_F16, "bf16": q8.Q8_TYPE_BF16}[kind]
        page_bytes = q8.q8_kv_page_bytes(code, page, kv, dim)
        pools = [np.full((layers, n_pages, page_bytes), 0xff, np.uint8) for _ in range(2)]   # NaNs, quants of -1
        for i, n in enumerate(lens):
            both = []
            for w in range(2):
                x = rng.standard_normal((n, kv, dim)).astype(np.float32) * (v_scale if w else 1.0)
                if n > 3:
                    x[n // 2, :, : dim // 2] = 0.0                   # all-zero blocks
                if kind == "q8":
                    qv, d = dequantise(x, dim)
                    exact = qv.astype(np.float64) * np.repeat(d.astype(np.float64), 32, -1)
                else:
                    t = torch.from_numpy(x).to(DT[kind])
                    exact, raw = f64(t), (t.view(torch.uint8).numpy() if n else None)
                both.append(exact)
                for j in range(n):
                    pg = pools[w][layer, table[i, j // page]].reshape(kv, -1)
                    r = j % page
                    if kind == "q8":
                        pg[:, r * dim:(r + 1) * dim] = qv[j].view(np.uint8)
                        o = page * dim + r * (dim // 16)
                        pg[:, o:o + dim // 16] = d[j].view(np.uint8)
                    else:
                        pg[:, r * dim * 2:(r + 1) * dim * 2] = raw[j]
            self.rows.append(both)
        k, v = (torch.from_numpy(x) for x in pools)
        if strided:                                                  # K and V of a page side by side, and a gap
            both = torch.full((layers, n_pages, 2 * page_bytes + 64), 0xff, dtype=torch.uint8)
            both[..., :page_bytes], both[..., page_bytes:2 * page_bytes] = k, v
            both = both.to(DEV)
            k, v = both[..., :page_bytes], both[..., page_bytes:2 * page_bytes]
        else:
            k, v = k.to(DEV), v.to(DEV)
        self.cache = q8.KVCache(k, v, code, page, kv, dim)
        self.table = torch.from_numpy(table).to(DEV)
        self.lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)


def check(got, ref, bound, what):
    err = np.abs(got - ref)
    assert not np.isnan(got).any(), f"{what}: NaN"
    assert np.all(err <= bound), f"{what}: {np.max(err / bound):.2f} of the bound, worst at {np.unravel_index(np.argmax(err / bound), err.shape)}"


def check_decode(q8, kind, lens, heads, kv, dim, page, qtype=None, window=0, sinks=False, seed=0, out=None, **kw):
    qtype = qtype or ("f16" if kind == "q8" else kind)
    layers = kw.get("layers", 1)
    pool = Pool(q8, kind, lens, kv, dim, page, seed + 1, **kw)
    rng = np.random.default_rng(seed)
    n = len(lens)
    fused = torch.from_numpy(rng.standard_normal((n, heads + 3, dim)).astype(np.float32)).to(DT[qtype]).to(DEV)
    q = fused[:, 1:1 + heads]                                        # rows strided
    sk = torch.from_numpy(rng.standard_normal(heads).astype(np.float32)).to(DEV) if sinks else None
    code = {None: None, "f32": q8.Q8_TYPE_F32, "q8": q8.Q8_TYPE_Q8_0}[out]
    o, lse = q8.attn_decode(q, pool.cache, kw.get("layer", 0), pool.table, pool.lens_t, window=window, sinks=sk,
                            out_type=code, want_lse=True)
    assert q8.q8_last_error() == 0
    if out == "q8":
        o32 = q8.attn_decode(q, pool.cache, kw.get("layer", 0), pool.table, pool.lens_t, window=window, sinks=sk,
                             out_type=q8.Q8_TYPE_F32)
        assert torch.equal(o.view(n, -1), q8.quantize_act(o32.view(n, -1)))
        return
    got, got_lse = f64(o), f64(lse)
    for i, m in enumerate(lens):
        for h in range(heads):
            k, v = (x[:, h // (heads // kv)] for x in pool.rows[i])
            see = np.zeros((1, m), bool)
            see[0, max(0, m - window) if window else 0:] = True
            r, rl, b, bl = attend(f64(q[i, h])[None], k, v, see, dim ** -0.5, None if sk is None else float(sk[h]),
                                  "bf16" if kind == "bf16" else "f16", out or qtype)
            check(got[i, h][None], r, b, f"seq {i} (len {m}) head {h}")
            if rl[0] == -np.inf:
                assert got_lse[i, h] == -np.inf
            else:
                assert abs(got_lse[i, h] - rl[0]) <= bl[0], f"lse of seq {i} head {h}"
    again = q8.attn_decode(q, pool.cache, kw.get("layer", 0), pool.table, pool.lens_t, window=window, sinks=sk, out_type=code)
    assert torch.equal(o, again), "not the same bits on a second run"


@pytest.mark.parametrize("kind", ["bf16", "f16", "q8"])
@pytest.mark.parametrize("dim", [64, 128, 256, 512])
def test_decode_lengths(q8, kind, dim):
    """Empty and one-token sequences, lengths around the tile sizes and page ends."""
    check_decode(q8, kind, [0, 1, 15, 16, 17, 63, 64, 65, 130, 257], heads=4, kv=2, dim=dim, page=16, seed=dim)


@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 8), (9, 3), (16, 2), (20, 1), (28, 4), (64, 1)])
@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_decode_head_layouts(q8, kind, heads, kv):
    check_decode(q8, kind, [33, 100, 0, 7], heads=heads, kv=kv, dim=128 if heads < 64 else 64, page=32, seed=heads)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kind,dim", [("f16", 128), ("q8", 64), ("q8", 512), ("bf16", 512)])
def test_decode_pages(q8, kind, dim, page):
    check_decode(q8, kind, [300, 255, 5], heads=4, kv=1, dim=dim, page=page, seed=page, sinks=True)


@pytest.mark.parametrize("window", [1, 16, 37, 100, 5000])
@pytest.mark.parametrize("kind", ["bf16", "q8"])
def test_decode_window_and_sinks(q8, kind, window):
    check_decode(q8, kind, [0, 1, 36, 37, 38, 200, 333], heads=6, kv=2, dim=128, page=16, window=window, sinks=True,
                 seed=window)


def test_decode_q8_with_bf16_queries(q8):
    check_decode(q8, "q8", [70, 3, 129], heads=8, kv=2, dim=128, page=32, qtype="bf16")
    check_decode(q8, "q8", [70, 3, 129], heads=8, kv=2, dim=64, page=32, qtype="bf16", sinks=True)


@pytest.mark.parametrize("v_scale", [1e-4, 300.0])
def test_decode_q8_value_scales(q8, v_scale):
    """Block scales far from 1: weights that carry them neither overflow nor vanish in fp16."""
    check_decode(q8, "q8", [200, 65], heads=8, kv=1, dim=128, page=32, v_scale=v_scale)


def test_decode_many_splits_and_rows(q8):
    """A long sequence over many CTAs beside short ones, and more sequences than threads of a CTA."""
    check_decode(q8, "bf16", [9000, 40, 3], heads=4, kv=1, dim=64, page=64)
    check_decode(q8, "f16", [int(x) for x in np.random.default_rng(5).integers(0, 40, 300)], heads=2, kv=1, dim=64, page=16)


def test_decode_strided_pool_and_layers(q8):
    check_decode(q8, "f16", [50, 129], heads=4, kv=2, dim=128, page=32, strided=True, layers=3, layer=2)
    check_decode(q8, "q8", [50, 129], heads=4, kv=2, dim=64, page=16, strided=True, layers=2, layer=1)


@pytest.mark.parametrize("out", ["f32", "q8"])
@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("q8", 64), ("f16", 512)])
def test_decode_output_types(q8, kind, dim, out):
    check_decode(q8, kind, [70, 0, 300], heads=3, kv=1, dim=dim, page=32, out=out)


def test_decode_bad_pages_and_lengths(q8):
    """A page id outside the pool leaves its positions out; lengths are cut to the table; both are reported."""
    pool = Pool(q8, "bf16", [100, 64], 2, 128, 32, 3)
    q = torch.randn(2, 4, 128, device=DEV).bfloat16()
    good = q8.attn_decode(q, pool.cache, 0, pool.table, pool.lens_t)
    for bad in (-1, pool.cache.struct.n_pages, 1 << 30):
        t = pool.table.clone()
        t[0, 3] = bad                                                # positions 96 .. 99
        o = q8.attn_decode(q, pool.cache, 0, t, pool.lens_t)
        assert q8.q8_last_error() == q8.Q8_ERANGE
        ref = q8.attn_decode(q, pool.cache, 0, pool.table, torch.tensor([96, 64], dtype=torch.int32, device=DEV))
        assert torch.allclose(o.float(), ref.float(), atol=2e-2) and torch.equal(o[1], good[1])
        assert q8.q8_last_error() == 0
    t = pool.table.clone()
    t[0] = -1
    o = q8.attn_decode(q, pool.cache, 0, t, torch.tensor([-5, 64], dtype=torch.int32, device=DEV))
    assert torch.all(o[0] == 0) and q8.q8_last_error() == q8.Q8_ERANGE
    lens = torch.tensor([1 << 30, 64], dtype=torch.int32, device=DEV)
    o = q8.attn_decode(q, pool.cache, 0, t, lens)                    # cut to the table, every page bad
    assert torch.all(o[0] == 0) and torch.equal(o[1], good[1]) and q8.q8_last_error() == q8.Q8_ERANGE


@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 128), (24, 1, 512)])
def test_decode_beyond_four_gigabytes(q8, heads, kv, dim):
    """Pages whose offsets pass 32 bits, by decode, append and the page copies."""
    page, n = 64, 150
    page_bytes = q8.q8_kv_page_bytes(q8.Q8_TYPE_F16, page, kv, dim)
    n_pages = (5 << 30) // page_bytes
    cache = q8.KVCache(*(torch.empty((1, n_pages, page_bytes), dtype=torch.uint8, device=DEV) for _ in range(2)),
                       q8.Q8_TYPE_F16, page, kv, dim)
    table = torch.tensor([[n_pages - 1, n_pages - 7, n_pages - 2]], dtype=torch.int32, device=DEV)
    small = q8.KVCache.empty(q8.Q8_TYPE_F16, 1, 3, page, kv, dim)
    near = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    q, k, v = (torch.randn(n, h, dim, device=DEV) for h in (heads, kv, kv))
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    for c, t in ((cache, table), (small, near)):
        q16 = q8.kv_append(c, 0, q, k, v, pos, torch.zeros_like(pos), t)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    ref = q8.attn_decode(q16[-1:], small, 0, near, lens)
    assert torch.equal(q8.attn_decode(q16[-1:], cache, 0, table, lens), ref)
    moved = torch.tensor([[n_pages - 20, n_pages - 30, n_pages - 9]], dtype=torch.int32, device=DEV)
    q8.kv_copy(cache, table[0], moved[0])
    assert torch.equal(q8.attn_decode(q16[-1:], cache, 0, moved, lens), ref) and q8.q8_last_error() == 0


def test_decode_thousands_of_sequences(q8):
    """Rows of many short sequences against the same rows one call each."""
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(0, 20, 3000)]
    pool = Pool(q8, "bf16", lens, 1, 64, 16, 9)
    q = torch.randn(3000, 2, 64, device=DEV).bfloat16()
    o = q8.attn_decode(q, pool.cache, 0, pool.table, pool.lens_t)
    for i in (0, 1, 17, 1500, 2998, 2999):
        one = q8.attn_decode(q[i:i + 1], pool.cache, 0, pool.table[i:i + 1], pool.lens_t[i:i + 1])
        assert torch.equal(one[0], o[i])
    assert q8.q8_last_error() == 0


def test_decode_in_a_graph_and_on_a_stream(q8):
    pool = Pool(q8, "bf16", [300, 64, 0, 17], 2, 128, 32, 4)
    q = torch.randn(4, 8, 128, device=DEV).bfloat16()
    ref = q8.attn_decode(q, pool.cache, 0, pool.table, pool.lens_t)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        a = q8.attn_decode(q, pool.cache, 0, pool.table, pool.lens_t)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(a, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b = q8.attn_decode(q, pool.cache, 0, pool.table, pool.lens_t)
    for _ in range(3):
        b.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b, ref)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [256, 512])
@pytest.mark.parametrize("heads,kv", [(64, 1), (17, 1), (40, 2), (130, 2)])
def test_decode_many_heads_on_one(q8, kind, dim, heads, kv):
    """More than 16 query heads on a key-value head: the tcgen05 kernel, with full, part and several head tiles."""
    check_decode(q8, kind, [0, 1, 127, 128, 129, 300], heads=heads, kv=kv, dim=dim, page=32, seed=heads, sinks=heads != 64)


@pytest.mark.parametrize("page", [16, 64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 50, 130])
def test_decode_many_heads_pages_and_windows(q8, page, window):
    check_decode(q8, "f16", [700, 131, 0, 16], heads=20, kv=1, dim=512, page=page, window=window, seed=page + window, strided=True,
                 layers=2, layer=1)


@pytest.mark.parametrize("out", ["f32", "q8"])
def test_decode_many_heads_output_types(q8, out):
    check_decode(q8, "bf16", [70, 0, 300], heads=33, kv=1, dim=512, page=32, out=out)


def test_decode_many_heads_long(q8):
    """Units over many CTAs, and more sequences than CTAs."""
    check_decode(q8, "bf16", [6000, 5, 900], heads=18, kv=1, dim=256, page=64)
    check_decode(q8, "f16", [int(x) for x in np.random.default_rng(6).integers(0, 30, 170)], heads=17, kv=1, dim=256, page=16)


def test_decode_many_heads_growing_scores(q8):
    """Scores that rise along the sequence: the running maxima move in many steps."""
    pool = Pool(q8, "f16", [900], 1, 512, 32, 8)
    q = torch.randn(1, 24, 512, device=DEV).half()
    k = pool.cache.k.view(torch.float16).view(1, -1, 1, 32, 512)
    ramp = torch.linspace(-1.0, 1.0, 900)
    row = (q[0, 0].float().cpu() * 0.06)
    for j in range(900):
        k[0, int(pool.table[0, j // 32]), 0, j % 32] = (row * ramp[j] * 8).half().to(DEV)
    keys = f64(k[0, pool.table[0, :29].long()])[:, 0].reshape(-1, 512)[:900]
    got = f64(q8.attn_decode(q, pool.cache, 0, pool.table, pool.lens_t))
    assert q8.q8_last_error() == 0
    for h in range(24):
        r, _, b, _ = attend(f64(q[0, h])[None], keys, pool.rows[0][1][:, 0], np.ones((1, 900), bool), 512 ** -0.5, None, "f16", "f16")
        check(got[0, h][None], r, b, f"head {h}")


def test_decode_many_heads_bad_pages(q8):
    pool = Pool(q8, "bf16", [200, 64], 1, 512, 32, 3)
    q = torch.randn(2, 24, 512, device=DEV).bfloat16()
    good = q8.attn_decode(q, pool.cache, 0, pool.table, pool.lens_t)
    for bad in (-1, pool.cache.struct.n_pages, 1 << 30):
        t = pool.table.clone()
        t[0, 6] = bad                                                # positions 192 .. 199
        o = q8.attn_decode(q, pool.cache, 0, t, pool.lens_t)
        assert q8.q8_last_error() == q8.Q8_ERANGE
        ref = q8.attn_decode(q, pool.cache, 0, pool.table, torch.tensor([192, 64], dtype=torch.int32, device=DEV))
        assert torch.equal(o[0], ref[0]) and torch.equal(o[1], good[1])
    o = q8.attn_decode(q, pool.cache, 0, torch.full_like(pool.table, -1), pool.lens_t)
    assert torch.all(o == 0) and q8.q8_last_error() == q8.Q8_ERANGE


def test_decode_many_heads_wait_expires(q8):
    """The tcgen05 decode kernel with its producer withholding every copy reports Q8_ETIMEOUT and returns."""
    pool = Pool(q8, "bf16", [200, 64], 1, 512, 32, 3)
    q = torch.randn(2, 24, 512, device=DEV).bfloat16()
    ref = q8.attn_decode(q, pool.cache, 0, pool.table, pool.lens_t)
    assert q8.q8_last_error() == 0
    q8.q8_debug_expire_waits(1, 1_000_000)
    q8.attn_decode(q, pool.cache, 0, pool.table, pool.lens_t)
    assert q8.q8_last_error() == q8.Q8_ETIMEOUT
    assert torch.equal(q8.attn_decode(q, pool.cache, 0, pool.table, pool.lens_t), ref)
    assert q8.q8_last_error() == 0


@pytest.mark.parametrize("kind,dim,heads,kv", [("f16", 64, 16, 1), ("bf16", 128, 3, 1), ("q8", 128, 4, 2), ("q8", 512, 2, 1)])
def test_decode_pieces_joined_in_groups(q8, kind, dim, heads, kv):
    """Few units over all CTAs: their pieces are joined in groups, with sequences of a few tiles and of none beside."""
    check_decode(q8, kind, [21000, 0, 70, 9001], heads=heads, kv=kv, dim=dim, page=64, seed=dim, sinks=True)
    check_decode(q8, kind, [30011], heads=heads, kv=kv, dim=dim, page=128, seed=dim + 1, window=25000)


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8"])
@pytest.mark.parametrize("dim", [64, 128, 256, 512])
def test_decode_whole_units(q8, kind, dim):
    """Short sequences only: CTAs take whole units, more of them than CTAs, empty ones among them."""
    rng = np.random.default_rng(dim)
    check_decode(q8, kind, [0, 1, 0, 63, 64, 65, 128, 0], heads=6, kv=2, dim=dim, page=16, seed=1, sinks=True)
    check_decode(q8, kind, [int(x) * int(x > 3) for x in rng.integers(0, 40, 330)], heads=2, kv=2, dim=dim, page=16, seed=2)
    check_decode(q8, kind, [0, 0, 0], heads=5, kv=1, dim=dim, page=16, seed=3)


@pytest.mark.parametrize("heads", [17, 64])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_decode_many_heads_little_room(q8, kind, heads):
    """More than 16 query heads on a key-value head with room for a few positions, or a window of a few."""
    check_decode(q8, kind, [0, 1, 40, 64], heads=heads, kv=1, dim=512, page=64, seed=heads, sinks=True)
    check_decode(q8, kind, [300, 0, 64, 1000], heads=heads, kv=1, dim=256, page=32, seed=heads, window=30)


# ------------------------------------------------------------------ whole prompts
def check_prompt(q8, kind, qlens, klens, heads, kv, dim, window=0, sinks=False, seed=0, out=None, poison=True):
    rng = np.random.default_rng(seed)
    dt = DT[kind]
    q0, k0 = np.concatenate([[0], np.cumsum(qlens)]), np.concatenate([[0], np.cumsum(klens)])

    def fused(n, h, extra):                                          # rows strided: heads inside a wider row
        x = torch.from_numpy(rng.standard_normal((n, h + extra, dim)).astype(np.float32)).to(dt).to(DEV)
        return x[:, extra:]

    q, kvt = fused(int(q0[-1]), heads, 2), fused(int(k0[-1]) + 200, 2 * kv, 1)
    kvt[int(k0[-1]):] = float("nan")                                 # rows of no sequence
    k, v = kvt[:, :kv], kvt[:, kv:]
    sk = torch.from_numpy(rng.standard_normal(heads).astype(np.float32)).to(DEV) if sinks else None
    code = {None: None, "f32": q8.Q8_TYPE_F32, "q8": q8.Q8_TYPE_Q8_0}[out]
    qs, ks = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (q0, k0))
    args = dict(window=window, sinks=sk)
    o, lse = q8.attn_prompt(q, k, v, qs, None if list(qlens) == list(klens) else ks, out_type=code, want_lse=True, **args)
    assert q8.q8_last_error() == 0
    if out == "q8":
        o32 = q8.attn_prompt(q, k, v, qs, ks, out_type=q8.Q8_TYPE_F32, **args)
        assert torch.equal(o.view(q.shape[0], -1), q8.quantize_act(o32.view(q.shape[0], -1)))
        return
    got, got_lse, kf, vf, qf = f64(o), f64(lse), f64(k), f64(v), f64(q)
    for s in range(len(qlens)):
        lq, lk = qlens[s], klens[s]
        last = np.arange(lq)[:, None] + lk - lq
        j = np.arange(lk)
        see = (j <= last) & ((j > last - window) if window else True)
        for h in range(heads):
            kk, vv = (x[k0[s]:k0[s + 1], h // (heads // kv)] for x in (kf, vf))
            r, rl, b, bl = attend(qf[q0[s]:q0[s + 1], h], kk, vv, see, dim ** -0.5, None if sk is None else float(sk[h]),
                                  kind, out or kind)
            check(got[q0[s]:q0[s + 1], h], r, b, f"seq {s} ({lq}, {lk}) head {h}")
            gl = got_lse[q0[s]:q0[s + 1], h]
            empty = rl == -np.inf
            assert np.all(gl[empty] == -np.inf) and np.all(np.abs(gl[~empty] - rl[~empty]) <= bl[~empty]), f"lse {s} {h}"
    again = q8.attn_prompt(q, k, v, qs, ks, out_type=code, **args)
    assert torch.equal(o, again), "not the same bits on a second run"


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256, 512])
def test_prompt_lengths(q8, kind, dim):
    lens = [1, 2, 63, 64, 65, 0, 127, 128, 129, 257]
    check_prompt(q8, kind, lens, lens, heads=2, kv=1, dim=dim, seed=dim)


@pytest.mark.parametrize("heads,kv", [(1, 1), (4, 4), (9, 3), (16, 2), (20, 1)])
def test_prompt_head_layouts(q8, heads, kv):
    check_prompt(q8, "bf16", [70, 130], [70, 130], heads=heads, kv=kv, dim=128, seed=heads)


@pytest.mark.parametrize("dim", [64, 128, 512])
def test_prompt_prefix_and_short_keys(q8, dim):
    """Cached prefixes (more keys than queries), fewer keys than queries (the first rows see nothing), no keys."""
    check_prompt(q8, "f16", [5, 100, 64, 300, 7], [205, 130, 30, 1, 0], heads=2, kv=1, dim=dim, seed=dim)
    check_prompt(q8, "bf16", [300, 200], [100, 260], heads=2, kv=2, dim=dim, seed=dim, sinks=True)


@pytest.mark.parametrize("window", [1, 17, 64, 200, 5000])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_window_and_sinks(q8, dim, window):
    check_prompt(q8, "bf16", [300, 66, 1], [300, 150, 1], heads=2, kv=1, dim=dim, window=window, sinks=True, seed=window)


def test_prompt_without_any_key(q8):
    for dim in (64, 512):
        q = torch.randn(5, 2, dim, device=DEV).half()
        none = torch.empty(0, 1, dim, device=DEV, dtype=torch.float16)
        start, empty = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 2, 5], [0, 0, 0]))
        o, lse = q8.attn_prompt(q, none, none, start, empty, want_lse=True)
        assert torch.all(o == 0) and torch.all(lse == -float("inf")) and q8.q8_last_error() == 0


@pytest.mark.parametrize("dim", [64, 128, 256, 512])
def test_prompt_more_tiles_than_sms(q8, dim):
    """Persistent CTAs over the list of tiles: many sequences, empty ones among them, several tiles a CTA."""
    rng = np.random.default_rng(dim)
    lens = [int(x) for x in rng.integers(0, 300, 90)]
    keys = [n + int(e) for n, e in zip(lens, rng.integers(-40, 60, 90).clip(min=[-n for n in lens]))]
    check_prompt(q8, "bf16", lens, keys, heads=2, kv=1, dim=dim, seed=dim, window=200, sinks=True)


def test_prompt_thousands_of_sequences(q8):
    """Many sequences, one of them long, against the same sequences in calls of their own."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 6, 2500)
    lens[1234] = 2000
    start = np.concatenate([[0], np.cumsum(lens)])
    n = int(start[-1])
    q, k, v = (torch.randn(n, h, 64, device=DEV).half() for h in (4, 2, 2))
    st = torch.tensor(start, dtype=torch.int32, device=DEV)
    o = q8.attn_prompt(q, k, v, st)
    for s in (0, 5, 1234, 2400, 2499):
        a, b = int(start[s]), int(start[s + 1])
        if a < b:
            one = q8.attn_prompt(q[a:b], k[a:b], v[a:b], torch.tensor([0, b - a], dtype=torch.int32, device=DEV))
            assert (one.float() - o[a:b].float()).abs().max() <= 2.0 ** -9 * 5     # |v| < 5, weights rounded to 2^-11
    assert q8.q8_last_error() == 0


def test_prompt_growing_scores(q8):
    """Scores that rise along the sequence: outputs are rescaled in many key tiles."""
    for dim in (64, 128, 512):
        n = 1000
        g = torch.Generator().manual_seed(dim)
        q, v = (torch.randn((n, 1, dim), generator=g).half().to(DEV) for _ in range(2))
        ramp = torch.linspace(-1.0, 1.0, n).to(DEV)[:, None, None]
        k = (q[n // 2:n // 2 + 1].float() * ramp * 0.06 * 8).half()
        got = f64(q8.attn_prompt(q, k, v, torch.tensor([0, n], dtype=torch.int32, device=DEV)))
        see = np.tril(np.ones((n, n), bool))
        r, _, b, _ = attend(f64(q)[:, 0], f64(k)[:, 0], f64(v)[:, 0], see, dim ** -0.5, None, "f16", "f16")
        check(got[:, 0], r, b, f"dim {dim}")


def test_prompt_long(q8):
    check_prompt(q8, "bf16", [1500], [1500], heads=2, kv=1, dim=128, seed=1)
    check_prompt(q8, "f16", [1100, 40], [1300, 40], heads=2, kv=1, dim=64, seed=2, window=600)


@pytest.mark.parametrize("out", ["f32", "q8"])
@pytest.mark.parametrize("dim", [64, 128, 512])
def test_prompt_output_types(q8, dim, out):
    check_prompt(q8, "bf16", [70, 150], [70, 150], heads=3, kv=1, dim=dim, out=out)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 512])
@pytest.mark.parametrize("window", [0, 40])
def test_prompt_unseen_values_stay_out(q8, kind, dim, window):
    """A key and value that are not finite reach exactly the rows that see them."""
    n, bad = 300, 141
    g = torch.Generator().manual_seed(dim)
    q, k, v = (torch.randn((n, 2, dim), generator=g).to(DT[kind]).to(DEV) for _ in range(3))
    start = torch.tensor([0, 100, n], dtype=torch.int32, device=DEV)
    clean = q8.attn_prompt(q, k, v, start, window=window)
    sees = torch.arange(n) >= bad
    if window:
        sees &= torch.arange(n) < bad + window
    for what, val in (("k", float("nan")), ("v", float("nan")), ("v", float("inf")), ("v", float("-inf"))):
        k2, v2 = k.clone(), v.clone()
        (k2 if what == "k" else v2)[bad, 1, 3] = val
        o = q8.attn_prompt(q, k2, v2, start, window=window)
        assert q8.q8_last_error() == 0
        assert torch.equal(o[:, 0], clean[:, 0]) and torch.equal(o[~sees], clean[~sees]), (what, val)
        if what == "k":
            assert torch.isnan(o[sees][:, 1]).all()
        else:
            hit = o[sees][:, 1, 3].float().cpu()
            assert torch.isnan(hit).all() if val != val else torch.all(hit == val)
            rest = torch.arange(dim) != 3
            assert torch.equal(o[sees][:, 1][:, rest], clean[sees][:, 1][:, rest])


def test_prompt_bad_starts(q8):
    """Starts outside the rows are cut and reported; nothing outside is read or written."""
    q = torch.randn(50, 2, 64, device=DEV).half()
    kv = torch.randn(50, 2, 64, device=DEV).half()
    ok = q8.attn_prompt(q, kv, kv, torch.tensor([0, 20, 50], dtype=torch.int32, device=DEV))
    o = q8.attn_prompt(q, kv, kv, torch.tensor([-7, 20, 1 << 30], dtype=torch.int32, device=DEV))
    assert q8.q8_last_error() == q8.Q8_ERANGE and torch.equal(o, ok)
    q8.attn_prompt(q, kv, kv, torch.tensor([30, 10, 50], dtype=torch.int32, device=DEV))
    assert q8.q8_last_error() == q8.Q8_ERANGE


def test_decode_agrees_with_the_last_prompt_row(q8):
    """The same tokens as a prompt and as a cached sequence with one new token."""
    n, kv, heads, dim, page = 200, 2, 8, 128, 32
    q, k, v = (torch.randn((n, h, dim), device=DEV) for h in (heads, kv, kv))
    table = torch.arange(7, dtype=torch.int32, device=DEV).flip(0)[None].contiguous()
    cache = q8.KVCache.empty(q8.Q8_TYPE_BF16, 1, 7, page, kv, dim)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    q16, k16, v16 = q8.kv_append(cache, 0, q, k, v, pos, torch.zeros_like(pos), table, want_kv=True)
    start = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    a = q8.attn_prompt(q16, k16, v16, start, out_type=q8.Q8_TYPE_F32)[-1]
    b = q8.attn_decode(q16[-1:], cache, 0, table, torch.tensor([n], dtype=torch.int32, device=DEV), out_type=q8.Q8_TYPE_F32)[0]
    assert q8.q8_last_error() == 0
    # both within 2^-8 of the exact value in units of the weighted mean of |v| (below 1.2 for 200 normal values)
    assert (a - b).abs().max() <= 2 * 1.2 * 2.0 ** -8


def test_attn_prompt_wait_expires(q8):
    """The tcgen05 prompt attention with its producer withholding every copy: it reports Q8_ETIMEOUT, returns, and
    the next call is right again."""
    q = torch.randn(300, 2, 128, device=DEV).bfloat16()
    start = torch.tensor([0, 300], dtype=torch.int32, device=DEV)
    ref = q8.attn_prompt(q, q, q, start)
    assert q8.q8_last_error() == 0
    q8.q8_debug_expire_waits(1, 1_000_000)
    q8.attn_prompt(q, q, q, start)
    assert q8.q8_last_error() == q8.Q8_ETIMEOUT
    assert torch.equal(q8.attn_prompt(q, q, q, start), ref)
    assert q8.q8_last_error() == 0


@pytest.mark.parametrize("dim,tokens,heads", [(64, 300, 2), (64, 3000, 16), (256, 300, 2), (512, 150, 2)])
def test_attn_prompt_wait_expires_other_dims(q8, dim, tokens, heads):
    """The same for the kernels of the other head sizes, with one tile a CTA and with the list of tiles."""
    q = torch.randn(tokens, heads, dim, device=DEV).bfloat16()
    start = torch.tensor([0, tokens], dtype=torch.int32, device=DEV)
    ref = q8.attn_prompt(q, q, q, start)
    assert q8.q8_last_error() == 0
    q8.q8_debug_expire_waits(1, 1_000_000)
    q8.attn_prompt(q, q, q, start)
    assert q8.q8_last_error() == q8.Q8_ETIMEOUT
    assert torch.equal(q8.attn_prompt(q, q, q, start), ref)
    assert q8.q8_last_error() == 0
