"""Failure detection in q8_lora's tcgen05 kernels: with copies withheld their waits run out, the call ends promptly with
Q8_ETIMEOUT, and the next call is right."""
import time

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


def expired(q8, call):
    q8.q8_debug_expire_waits(1, 200_000)   # 0.2 ms instead of the normal 2 s
    try:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        call()
        assert q8.q8_last_error() == q8.Q8_ETIMEOUT
        assert time.perf_counter() - t0 < 0.5, "an expired wait did not end its kernel promptly"
    finally:
        q8.q8_debug_expire_waits(0, 0)


# outputs: whole tiles, a part of one (rows through the copy engine), rows that are not 16-byte aligned
@pytest.mark.parametrize("n,n_out", [(700, 4096), (3000, 8192), (700, 200), (2000, 1030)])
def test_copies_of_base(q8, n, n_out):
    """Tokens without an adapter: only the kernel of the outputs has work, which is to copy base."""
    g = torch.Generator(device=DEV).manual_seed(n)
    x, base = torch.randn(n, 64, generator=g, device=DEV), torch.randn(n, n_out, generator=g, device=DEV)
    a, b = (torch.zeros(2, *s, device=DEV, dtype=torch.bfloat16) for s in ((16, 64), (n_out, 16)))
    ids = torch.full((n,), -1, device=DEV, dtype=torch.int32)
    call = lambda: q8.lora(x, a, b, ids, base=base)
    assert torch.equal(call(), base) and q8.q8_last_error() == 0
    expired(q8, call)
    assert torch.equal(call(), base) and q8.q8_last_error() == 0


@pytest.mark.parametrize("n,n_in,n_out,rank,kind,x", [(700, 1024, 4096, 16, "bfloat16", "float32"), (3000, 1024, 512, 128, "float16", "float32"),
                                                      (2000, 4096, 1030, 96, "bfloat16", "float16"), (600, 16384, 256, 128, "bfloat16", "float32")])
def test_both_kernels(q8, n, n_in, n_out, rank, kind, x):
    """Both kernels, with whole sums and with sums in runs, x by the copy engine."""
    g = torch.Generator(device=DEV).manual_seed(n)
    xv = torch.randn(n, n_in, generator=g, device=DEV).to(getattr(torch, x))
    a, b = ((torch.randn(2, *s, generator=g, device=DEV) * s[1] ** -0.5).to(getattr(torch, kind)) for s in ((rank, n_in), (n_out, rank)))
    ids, base = torch.randint(0, 2, (n,), generator=g, device=DEV).int(), torch.randn(n, n_out, generator=g, device=DEV)
    call = lambda: q8.lora(xv, a, b, ids, base=base)
    want = call()
    assert q8.q8_last_error() == 0
    for _ in range(2):
        expired(q8, call)
    assert torch.equal(call(), want) and q8.q8_last_error() == 0
