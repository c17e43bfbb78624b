"""GPU tests of the page calls at the ends of their numbers, and with requests that break their rules."""
import pytest

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


@pytest.mark.parametrize("n_pages", [50, 1 << 24])
def test_reserve_sums_beyond_32_bits(q8, n_pages):
    """128 rows of 2^24 pages each: 2^31 pages, refused as a whole."""
    rows, width, page = 128, 1 << 24, 16
    cache = q8.KVCache.empty(q8.Q8_TYPE_Q8_0, 1, n_pages, page, 1, 64)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    lens, refs = torch.zeros(rows, dtype=torch.int32, device=DEV), torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    q8.kv_reserve(cache, table, lens, refs, i32(list(range(rows))), i32([width * page] * rows))
    assert q8.q8_last_error() == q8.Q8_ENOPAGE
    assert not lens.any() and not refs.any() and int(table.max()) == -1
    q8.kv_reserve(cache, table, lens, refs, i32([5, 9]), i32([33, 1]))
    assert q8.q8_last_error() == 0 and table[5, :4].tolist() == [0, 1, 2, -1] and table[9, :2].tolist() == [3, -1]
    del table
    torch.cuda.empty_cache()


def test_requests_that_name_a_row_twice_touch_nothing_else(q8):
    """Against the rules of q8.h: the rows and pages concerned may come out either way, all others stay."""
    page, n_pages, width, rows = 16, 40, 2, 6
    for _ in range(20):
        cache = q8.KVCache.empty(q8.Q8_TYPE_F16, 1, n_pages, page, 1, 64)
        wide = torch.full((rows + 4, width), 12345, dtype=torch.int32, device=DEV)      # rows beyond the table's
        wide[:rows] = -1
        counts = torch.full((n_pages + 64,), 777, dtype=torch.int32, device=DEV)
        counts[:n_pages] = 0
        table, refs, lens = wide[:rows], counts[:n_pages], torch.zeros(rows, dtype=torch.int32, device=DEV)
        q8.kv_reserve(cache, table, lens, refs, i32([0, 5]), i32([7, 5]))
        before = wide.clone()
        # each fits its row of 32 tokens alone, not after the other, and needs no page or one
        q8.kv_reserve(cache, table, lens, refs, i32([5, 5, 5, 5] * 8), i32([11, 8, 20, 27] * 8))
        assert q8.q8_last_error() in (0, q8.Q8_ERANGE)
        assert torch.equal(wide[:5], before[:5]) and torch.equal(wide[rows:], before[rows:])
        assert torch.all(counts[n_pages:] == 777) and int(table.max()) < n_pages and int(table.min()) >= -1
        assert 5 <= int(lens[5]) <= 32
        # a source that is overwritten by the same call
        q8.kv_fork(cache, table, lens, refs, i32([0, 5, 0]), i32([5, 1, 1]))
        assert q8.q8_last_error() in (0, q8.Q8_ERANGE)
        assert torch.equal(wide[0], before[0]) and torch.equal(wide[2:5], before[2:5]) and torch.equal(wide[rows:], before[rows:])
        assert torch.all(counts[n_pages:] == 777) and int(table.max()) < n_pages and int(table.min()) >= -1


def test_caches_on_the_host_are_refused(q8):
    """With everything else on the GPU; a pair of pools on different devices makes no cache."""
    c = q8.KVCache.empty(q8.Q8_TYPE_F16, 1, 4, 64, 2, 64, device="cpu")
    x, table, one, refs = torch.zeros(1, 2, 64, device=DEV), i32([[0, 1]]), i32([0]), i32([0] * 4)
    for call in (lambda: q8.attn_decode(x.half(), c, 0, table, one), lambda: q8.kv_append(c, 0, x, x, x, one, one, table),
                 lambda: q8.kv_reserve(c, table, one, refs, one, one), lambda: q8.kv_fork(c, table, one, refs, one, one),
                 lambda: q8.kv_free(c, table, one, refs, one), lambda: q8.kv_compact(c, table, one, refs),
                 lambda: q8.kv_copy(c, one, one)):
        with pytest.raises(TypeError, match="cache: pages on the GPU"):
            call()
    with pytest.raises(ValueError, match="device"):
        q8.KVCache(c.k.to(DEV), c.v, q8.Q8_TYPE_F16, 64, 2, 64)
    assert q8.q8_last_error() == 0
