"""The limit of tests/test_gpu_lora_sums.py tells fp32 accuracy from less (no GPU): the adapters' products with one part of the values left
out, in 64 bits otherwise, are beyond it, and a plain fp32 product is within."""
import numpy as np
import pytest

from tests.test_gpu_lora_sums import LIMIT


def bf16_terms(v, n):
    """The sum of the first n terms of 8 bits each that an fp32 value is split into."""
    v, total = v.astype(np.float32).copy(), np.zeros(v.shape)
    for _ in range(n):
        t = (v.view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)
        total += t
        v = v - t
    return total


def error(n_in, rank, kind, fault):
    rng = np.random.default_rng(n_in + rank)
    x = rng.standard_normal((64, n_in)).astype(np.float32)
    a, b = (rng.standard_normal(s) * s[1] ** -0.5 for s in ((rank, n_in), (96, rank)))
    if kind == "f16":
        a, b = a.astype(np.float16).astype(np.float64), b.astype(np.float16).astype(np.float64)
    else:
        a, b = bf16_terms(a, 1), bf16_terms(b, 1)
    want = (x.astype(np.float64) @ a.T) @ b.T
    if fault == "fp32":
        got = (x @ a.astype(np.float32).T) @ b.astype(np.float32).T
    else:
        low = bf16_terms(x, 2 if fault == "x" else 3) @ (bf16_terms(a, 1) if fault == "a" else a).T
        got = bf16_terms(low.astype(np.float32), 2 if fault == "low" else 3) @ (bf16_terms(b, 1) if fault == "b" else b).T
    return np.sqrt(np.mean((got - want) ** 2) / np.mean(want ** 2))


@pytest.mark.parametrize("n_in,rank", [(256, 16), (320, 48), (4096, 72), (512, 128), (16384, 128)])
@pytest.mark.parametrize("kind,fault", [("bf16", "x"), ("bf16", "low"), ("bf16", "none"), ("bf16", "fp32"), ("f16", "x"), ("f16", "low"), ("f16", "a"),
                                        ("f16", "b"), ("f16", "none"), ("f16", "fp32")])
def test_a_term_left_out_is_beyond_the_limit(n_in, rank, kind, fault):
    e = error(n_in, rank, kind, fault)
    assert e <= LIMIT if fault in ("none", "fp32") else e > 4 * LIMIT
