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
