"""GPU tests of the adapters' accuracy: the root mean square of the errors against 64 bits, for sums of every length.

Limit: 2^-20 of the adapters' part (its root mean square).  An addition in the tensor cores takes up to 2^-26 of the sum away,
always towards zero, so these add up: 16 in a run of the first product and 8 in the second (128 / 16), 24 in all, where an
fp16 weight's second term takes part 16 more: 2.4 to 3.6 2^-22 of the part.  The rounded additions (parts, runs, the scale, base)
fall to either side, half a step, 2^-24 of their sums, each: 2^-22 for 16 of them.  Together below 2^-20.  A value of which only 16
bits took part would be wrong by up to 2^-15 of its power of two, 2^-16.3 of the part in the mean: 13 times the limit."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DEV = "cuda:0"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
LIMIT = 2.0 ** -20


@pytest.fixture(scope="module")
def q8():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_quantized_matmul_gb300 import build
    build.build()
    import q8_quantized_matmul_gb300 as m
    torch.cuda.set_device(0)
    return m


def values(blocks):
    raw = blocks.view(blocks.shape[0], -1, 34)
    d = raw[:, :, :2].contiguous().view(torch.float16).double()
    return (raw[:, :, 2:].contiguous().view(torch.int8).double() * d).view(blocks.shape[0], -1)


def error(q8, n, n_in, n_out, rank, adapters, kind, x_type, seed=0):
    """Root mean square of the errors over that of the adapters' part."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x = rand(n, n_in)
    x = q8.quantize_act(x) if x_type == "q8" else x.to(DT[x_type])
    a, b = (rand(adapters, rank, n_in) * n_in ** -0.5).to(DT[kind]), (rand(adapters, n_out, rank) * rank ** -0.5).to(DT[kind])
    ids = torch.randint(0, adapters, (n,), generator=g, device=DEV)
    got = q8.lora(x, a, b, ids.int())
    assert q8.q8_last_error() == 0
    xv, want = values(x) if x_type == "q8" else x, torch.empty(n, n_out, dtype=torch.double, device=DEV)
    for i in range(adapters):
        t = ids == i
        want[t] = (xv[t].double() @ a[i].double().T) @ b[i].double().T
    return float((got.double() - want).square().mean().sqrt() / want.square().mean().sqrt())


# tokens, adapters: up to 15 tiles (clusters of 8), 16 to 36 and more tiles (clusters of 4 for ranks up to 96)
@pytest.mark.parametrize("n,adapters", [(40, 2), (600, 2), (2500, 3), (4900, 3)])
@pytest.mark.parametrize("n_in,rank", [(512, 128), (4096, 16), (4096, 72), (4096, 128), (8192, 64), (8224, 96), (8192, 128), (16384, 64), (16416, 80),
                                       (16384, 128), (65536, 16), (32768, 128)])
def test_sums_of_every_length(q8, n, adapters, n_in, rank):
    assert error(q8, n, n_in, 200, rank, adapters, "bf16", "f32") <= LIMIT


@pytest.mark.parametrize("kind,x", [("f16", "f32"), ("bf16", "q8"), ("f16", "q8"), ("bf16", "bf16"), ("f16", "bf16"), ("bf16", "f16"), ("f16", "f16")])
@pytest.mark.parametrize("n_in,rank", [(16384, 64), (16384, 96), (16384, 128)])
def test_long_sums_of_every_type(q8, kind, x, n_in, rank):
    assert error(q8, 4900, n_in, 200, rank, 3, kind, x) <= LIMIT
