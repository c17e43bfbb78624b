"""GPU tests of the paged key-value cache's upkeep: q8_kv_append bit for bit against its formula, and the page
calls against a plain model of tables, reference counts and page data."""
import numpy as np
import pytest

import oracle

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


def rotate(x, cs, mode):
    """fp32, every product and sum rounded on its own."""
    rot = cs.shape[1]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    y = x.copy()
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if mode == 1 else (slice(0, rot, 2), slice(1, rot, 2))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


@pytest.mark.parametrize("kind", ["bf16", "f16", "q8"])
@pytest.mark.parametrize("dim,rope,rot", [(64, 0, 0), (64, 1, 64), (128, 1, 48), (128, 2, 64), (256, 2, 16), (512, 1, 512)])
def test_append(q8, kind, dim, rope, rot):
    rng = np.random.default_rng(dim + rope)
    n, heads, kv, page = 37, 5, 3, 16
    x = rng.standard_normal((n, heads + 2 * kv, dim)).astype(np.float32)
    x[3] = 0.0
    x[4] *= 1e-30                                                    # block scales that underflow binary16
    t = torch.from_numpy(x).to(DEV)
    q, k, v = t[:, :heads], t[:, heads:heads + kv], t[:, heads + kv:]
    seq_of = rng.integers(0, 3, n).astype(np.int32)
    pos = np.zeros(n, np.int32)
    for s in range(3):
        pos[seq_of == s] = 5 + np.arange((seq_of == s).sum())
    seq_of[7] = -1                                                   # padding: not stored
    table = rng.permutation(15).astype(np.int32).reshape(3, 5)
    cs = rng.standard_normal((64, rot)).astype(np.float32) if rope else None
    code = {"q8": q8.Q8_TYPE_Q8_0, "f16": q8.Q8_TYPE_F16, "bf16": q8.Q8_TYPE_BF16}[kind]
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    cache = q8.KVCache.empty(code, 2, 15, page, kv, dim)
    for pool in (cache.k, cache.v):
        pool.fill_(0xaa)
    q16, k16, v16 = q8.kv_append(cache, 1, q, k, v, i32(pos), i32(seq_of), torch.from_numpy(table).to(DEV),
                                 None if cs is None else torch.from_numpy(cs).to(DEV), rope, want_kv=True)
    assert q8.q8_last_error() == 0 and q16.dtype == dt
    xr = x.copy()
    if rope:
        xr[:, :heads + kv] = rotate(x[:, :heads + kv], cs[pos], rope)
    want = torch.from_numpy(xr).to(dt)
    for got, ref in ((q16, want[:, :heads]), (k16, want[:, heads:heads + kv]), (v16, want[:, heads + kv:])):
        assert torch.equal(got.cpu().view(torch.int16), ref.contiguous().view(torch.int16))
    for pool, rows in ((cache.k, xr[:, heads:heads + kv]), (cache.v, xr[:, heads + kv:])):
        ref = np.full((2, 15, kv, pool.shape[2] // kv), 0xaa, np.uint8)
        for i in range(n):
            if seq_of[i] < 0:
                continue
            pg, r = ref[1, table[seq_of[i], pos[i] // page]], pos[i] % page
            for h in range(kv):
                if kind == "q8":
                    blocks = oracle.get().quantize(np.ascontiguousarray(rows[i, h][None])).reshape(-1, 34)
                    pg[h, r * dim:(r + 1) * dim] = blocks[:, 2:].reshape(-1)
                    o = page * dim + r * (dim // 16)
                    pg[h, o:o + dim // 16] = blocks[:, :2].reshape(-1)
                else:
                    pg[h, r * dim * 2:(r + 1) * dim * 2] = torch.from_numpy(rows[i, h]).to(dt).view(torch.uint8).numpy()
        assert np.array_equal(pool.cpu().numpy().reshape(ref.shape), ref)


def test_append_without_cache_or_queries(q8):
    k, v = torch.randn(9, 2, 64, device=DEV), torch.randn(9, 2, 64, device=DEV)
    pos = i32(range(9))
    q16, k16, v16 = q8.kv_append(None, 0, None, k, v, pos, None, None, want_kv=True, dtype=torch.float16)
    assert q16 is None and torch.equal(k16, k.half()) and torch.equal(v16, v.half())
    assert q8.q8_last_error() == 0


def test_append_reports_bad_indices(q8):
    cache = q8.KVCache.empty(q8.Q8_TYPE_F16, 1, 4, 16, 1, 64)
    x = torch.randn(2, 1, 64, device=DEV)
    cs = torch.randn(40, 64, device=DEV)

    def call(pos, seq, table, rope=0):
        cache.k.zero_()
        q = q8.kv_append(cache, 0, x, x, x, i32(pos), i32(seq), i32(table), cs if rope else None, rope)
        return q, q8.q8_last_error(), int((cache.k[0].view(torch.float16).view(4, 16, 64).abs().sum(-1) > 0).sum())

    assert call([0, 17], [0, 0], [[0, 1]])[1:] == (0, 2)
    assert call([0, 32], [0, 0], [[0, 1]])[1:] == (q8.Q8_ERANGE, 1)      # beyond the row's pages
    assert call([0, -1], [0, 0], [[0, 1]])[1:] == (q8.Q8_ERANGE, 1)
    assert call([0, 17], [0, 1], [[0, 1]])[1:] == (q8.Q8_ERANGE, 1)      # no such row
    assert call([0, 17], [0, 0], [[0, 4]])[1:] == (q8.Q8_ERANGE, 1)      # no such page
    assert call([0, 17], [0, 0], [[0, -1]])[1:] == (q8.Q8_ERANGE, 1)
    assert call([0, 17], [0, -1], [[0, 1]])[1:] == (0, 1)                # padding is no error
    q, rc, stored = call([0, 40], [0, 0], [[0, 1, 2]], rope=1)           # no such angle: zeros, not stored
    assert (rc, stored) == (q8.Q8_ERANGE, 1) and torch.all(q[1] == 0) and torch.any(q[0] != 0)


class Model:
    """Tables, counts and page contents on the host."""

    def __init__(self, q8, n_pages, page, rows, width, layers=2, kv=2, dim=64, seed=0):
        rng = np.random.default_rng(seed)
        self.q8, self.page = q8, page
        shape = (layers, n_pages, kv * page * dim * 2)
        self.pools = [rng.integers(0, 256, shape).astype(np.uint8) for _ in range(2)]
        self.cache = q8.KVCache(*(torch.from_numpy(p).to(DEV) for p in self.pools), q8.Q8_TYPE_F16, page, kv, dim)
        self.pools = [p.copy() for p in self.pools]
        self.table = np.full((rows, width), -1, np.int32)
        self.lens, self.refs = np.zeros(rows, np.int32), np.zeros(n_pages, np.int32)
        self.up()

    def up(self):
        self.d = [torch.from_numpy(x.copy()).to(DEV) for x in (self.table, self.lens, self.refs)]

    def check(self, err=0):
        assert self.q8.q8_last_error() == err
        for name, a, b in zip(("table", "lens", "refs"), self.d, (self.table, self.lens, self.refs)):
            assert np.array_equal(a.cpu().numpy(), b), name
        for a, b in zip((self.cache.k, self.cache.v), self.pools):
            assert np.array_equal(a.cpu().numpy(), b), "page data"

    def free_pages(self):
        return list(np.flatnonzero(self.refs == 0))

    def reserve(self, rows, new, go=True):
        self.q8.kv_reserve(self.cache, *self.d, i32(rows), i32(new))
        if not go:
            return
        free = self.free_pages()
        for r, m in zip(rows, new):
            if r < 0:
                continue
            had, now = -(-self.lens[r] // self.page), -(-(self.lens[r] + m) // self.page)
            for s in range(had, now):
                self.table[r, s] = free.pop(0)
                self.refs[self.table[r, s]] = 1
            self.lens[r] += m

    def fork(self, src, dst, go=True):
        self.q8.kv_fork(self.cache, *self.d, i32(src), i32(dst))
        if not go:
            return
        free = self.free_pages()
        for a, b in zip(src, dst):
            if a < 0 or b < 0:
                continue
            whole, part = divmod(int(self.lens[a]), self.page)
            self.table[b] = -1
            self.table[b, :whole] = self.table[a, :whole]
            for p in self.table[a, :whole]:
                self.refs[p] += 1
            if part:
                p = free.pop(0)
                self.refs[p] = 1
                self.table[b, whole] = p
                for pool in self.pools:
                    pool[:, p] = pool[:, self.table[a, whole]]
            self.lens[b] = self.lens[a]

    def free(self, rows):
        self.q8.kv_free(self.cache, *self.d, i32(rows))
        for r in rows:
            if r < 0:
                continue
            for p in self.table[r, :-(-self.lens[r] // self.page)]:
                self.refs[p] -= 1
            self.table[r], self.lens[r] = -1, 0

    def compact(self):
        t, refs, used = self.q8.kv_compact(self.cache, *self.d)
        n = int((self.refs > 0).sum())
        at = np.arange(len(self.refs))
        holes, movers = at[(self.refs == 0) & (at < n)], at[(self.refs > 0) & (at >= n)]
        to = dict(zip(movers, holes))
        for pool in self.pools:
            pool[:, holes] = pool[:, movers]
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = np.vectorize(lambda p: to.get(p, p), otypes=[np.int32])(self.table)
        assert int(used) == n
        self.d = [t, self.d[1], refs]


@pytest.mark.parametrize("page", [16, 32, 256])
def test_pages_life(q8, page):
    """Grow, fork, free, fork again, compact, grow on, against the model after every step."""
    m = Model(q8, 60, page, 10, 8, seed=page)
    m.reserve([0, 3, -1, 7], [page + 5, 2 * page, 9, 1])
    m.check()
    m.fork([0, 3, 0, 7, -1], [1, 2, 4, 8, 9])
    m.check()
    m.reserve([0, 1, 5], [1, page, 0])
    m.check()
    m.free([0, 8, -1])
    m.check()
    m.fork([1, 1], [0, 8])
    m.check()
    m.free([3, 4])
    m.compact()
    m.check()
    m.reserve([3, 9], [3 * page, 5])
    m.check()
    m.free(list(range(10)))
    m.check()
    assert not m.refs.any()
    m.compact()
    m.check()


def test_pages_many_requests(q8):
    """More requests and pages than threads of the planning CTA."""
    m = Model(q8, 9000, 16, 3001, 3, layers=1, kv=1, seed=1)
    rng = np.random.default_rng(2)
    m.reserve(list(rng.permutation(1500)), [int(x) for x in rng.integers(0, 48, 1500)])
    m.check()
    m.fork(list(range(1500)), list(range(1500, 3000)))
    m.check()
    m.free([int(x) for x in rng.permutation(3000)[:1700]])
    m.check()
    m.compact()
    m.check()


def test_pages_run_out(q8):
    """All or nothing: a call that needs more pages than are free, or a longer row, changes nothing."""
    m = Model(q8, 6, 16, 5, 4)
    m.reserve([0, 1], [40, 20])                                      # 3 + 2 of 6 pages
    m.check()
    m.reserve([2, 3], [16, 1], go=False)                             # 2 needed, 1 free
    m.check(q8.Q8_ENOPAGE)
    m.fork([0, 1], [2, 3], go=False)
    m.check(q8.Q8_ENOPAGE)
    m.reserve([2, 1], [5, 60], go=False)                             # 80 tokens in a row of 64
    m.check(q8.Q8_ENOPAGE)
    m.reserve([2], [16])
    m.check()
    m.fork([2], [3])                                                 # whole pages need no new page
    m.check()


def test_pages_bad_rows(q8):
    m = Model(q8, 8, 16, 3, 4)
    m.reserve([0, 1], [20, 5])
    m.check()
    q8.kv_free(m.cache, *m.d, i32([3]))
    m.check(q8.Q8_ERANGE)
    q8.kv_fork(m.cache, *m.d, i32([0, 99]), i32([7, 2]))
    m.check(q8.Q8_ERANGE)
    q8.kv_reserve(m.cache, *m.d, i32([5, 0]), i32([1, -2]))
    m.check(q8.Q8_ERANGE)


def test_copy(q8):
    m = Model(q8, 12, 64, 2, 2, layers=3)
    q8.kv_copy(m.cache, i32([4, 7, -1, 4, 2, 99]), i32([0, 11, 3, 5, -1, 6]))
    for pool in m.pools:
        pool[:, 0], pool[:, 11], pool[:, 5] = pool[:, 4], pool[:, 7], pool[:, 4]
    m.check(q8.Q8_ERANGE)
