"""The example decoder: packed prefill, forks, single-token steps, release and compaction of a paged cache give the
hidden states of the whole sequences.

The two ways differ by the attention's rounding of its weights (2^-8 of a weighted mean of |v|, bf16) and the Q8_0
rounding of its output (half of 1/127 of a block's maximum), both below 2^-7 of the attention's output, which is one of
two terms added to the residual stream in each of two layers, and by quants of the following activations that fall
on another side (as much again): 4 x 2^-7 < 3.2e-2 of the stream.  A Q8_0 cache adds its keys' and values'
rounding, at most 1/254 of a block's maximum each: 2^-6 more in each layer."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("kind,most", [("Q8_TYPE_BF16", 3.2e-2), ("Q8_TYPE_Q8_0", 6.4e-2)])
def test_cached_decoder(kind, most):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from q8_quantized_matmul_gb300 import build
    build.build()
    import q8_quantized_matmul_gb300 as q8
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "cached_decoder.py")
    spec = importlib.util.spec_from_file_location("cached_decoder", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    worst = m.run(getattr(q8, kind))
    assert 0 <= worst <= most
