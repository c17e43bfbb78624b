"""What the calls around a layer's projections write in place is seen by autograd: a backward pass that needs the old values is
refused, where it would else take the new ones in silence."""
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


def lora_out(q8, t):
    a, b = torch.ones(1, 8, 64, device=DEV).bfloat16(), torch.ones(1, 64, 8, device=DEV).bfloat16()
    return q8.lora(torch.ones(t.shape[0], 64, device=DEV), a, b, torch.zeros(t.shape[0], dtype=torch.int32, device=DEV), base=t, out=t)


def norm_out(q8, t):
    return q8.residual_norm(t, torch.ones_like(t), None, 1e-6, h_out=t)[1]


def read_out(q8, t):
    cache = q8.KVCache.empty(q8.Q8_TYPE_BF16, 1, 1, 16, 1, 64)
    for pool in (cache.k, cache.v):
        pool.zero_()
    rows, table = t.view(-1, 1, 64), torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    start = torch.tensor([0, t.shape[0]], dtype=torch.int32, device=DEV)
    return q8.kv_read(cache, 0, table, start, t.shape[0], out=(rows, torch.empty_like(rows)))[0]


@pytest.mark.parametrize("call", [lora_out, norm_out, read_out])
def test_a_tensor_written_in_place_counts_as_changed(q8, call):
    x = torch.zeros(5, 64, device=DEV, requires_grad=True)
    t = x.exp()                                   # its gradient needs t
    with torch.no_grad():
        call(q8, t)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        t.sum().backward()
    t = x + 1                                     # this one's does not
    with torch.no_grad():
        call(q8, t)
    t.sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x))


@pytest.mark.parametrize("call", [lora_out, norm_out, read_out])
def test_inference_tensors(q8, call):
    with torch.inference_mode():
        t = torch.zeros(5, 64, device=DEV)
        call(q8, t)
    call(q8, t)
    assert q8.q8_last_error() == 0


def test_results_carry_no_gradients(q8):
    w = [torch.nn.Parameter(torch.ones(s, device=DEV).bfloat16()) for s in ((1, 8, 64), (1, 64, 8))]
    x = torch.ones(3, 64, device=DEV, requires_grad=True)
    out = q8.lora(x, *w, torch.zeros(3, dtype=torch.int32, device=DEV))
    assert not out.requires_grad and torch.equal(out, torch.full_like(out, 512))
