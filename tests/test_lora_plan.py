"""Which path a call of q8_lora takes (csrc/q8_lora_plan.h, compiled as plain C++), held to measured times of both."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "q8_quantized_matmul_gb300", "csrc")
SOURCE = """
#include "q8_lora_plan.h"
extern "C" int few(unsigned long long n, unsigned rank, unsigned long long n_in, unsigned long long n_out, unsigned adapters) {
    return q8::lora_few(n, rank, n_in, n_out, adapters, 152);
}
extern "C" unsigned splits(unsigned n, unsigned n_out) { return q8::lora_splits(n, n_out, 152); }
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    so = str(d / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fPIC", "-shared", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error", "-I", CSRC,
                    str(d / "plan.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.few.argtypes = [ctypes.c_uint64, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_uint64, ctypes.c_uint32]
    return lib


# inputs, outputs, rank, tokens, adapters (all in use), us of the few tokens' path and of the many tokens' path
MEASURED = [
    (1024, 32768, 32, 128, 1, 31.8, 21.9), (1024, 32768, 128, 32, 1, 39.0, 20.6), (1024, 32768, 128, 24, 1, 31.2, 20.7), (1024, 32768, 64, 64, 1, 33.3, 19.8),
    (1024, 32768, 64, 48, 1, 27.3, 19.6), (2048, 16384, 128, 32, 1, 34.0, 21.8), (8192, 8192, 128, 32, 1, 60.8, 37.0), (14336, 4096, 128, 32, 1, 92.0, 52.2),
    (8192, 8192, 128, 32, 2, 60.8, 34.3),
    (2048, 1000, 128, 48, 48, 14.6, 24.0), (2048, 1000, 128, 64, 64, 18.7, 27.6), (256, 512, 128, 48, 48, 11.3, 20.5),
    (4096, 4096, 16, 1, 8, 3.8, 20.0), (4096, 4096, 16, 64, 64, 6.9, 15.6), (4096, 4096, 16, 192, 192, 24.0, 33.7), (4096, 4096, 32, 128, 128, 23.2, 30.5),
    (4096, 4096, 16, 64, 1, 8.2, 24.0), (4096, 4096, 128, 32, 32, 27.0, 62.7), (4096, 4096, 128, 64, 1, 37.9, 28.1), (4096, 4096, 64, 96, 1, 33.3, 26.8),
    (1024, 32768, 32, 32, 40, 21.0, 88.0), (1024, 32768, 32, 128, 32, 38.9, 88.9), (1024, 32768, 16, 128, 128, 36.6, 45.8), (2048, 1000, 64, 333, 12, 60.0, 23.5)]


@pytest.mark.parametrize("n_in,n_out,rank,n,adapters,few,many", MEASURED)
def test_the_path_taken_is_the_quicker_one(plan, n_in, n_out, rank, n, adapters, few, many):
    assert (few if plan.few(n, rank, n_in, n_out, adapters) else many) <= 1.1 * min(few, many)


@pytest.mark.parametrize("n_in,n_out", [(32, 1), (1024, 32768), (1 << 31, 1), (32, (1 << 30) - 1), (65536, 65536)])
def test_calls_that_are_promised_no_scratch(plan, n_in, n_out):
    """At most 192 tokens, tokens times rank at most 4096, a quarter as many adapters as tokens: whatever the sizes."""
    for rank in range(8, 129, 8):
        for n in range(1, min(192, 4096 // rank) + 1):
            assert plan.few(n, rank, n_in, n_out, -(-n // 4)) and plan.few(n, rank, n_in, n_out, 16384)


def test_the_ends_of_the_range(plan):
    for n_in, n_out in ((32, 1), (1 << 31, 1), (32, (1 << 30) - 1), (4096, 4096)):
        assert not plan.few(193, 8, n_in, n_out, 16384) and not plan.few((1 << 31) - 1, 128, n_in, n_out, 1)
        assert plan.few(1, 8, n_in, n_out, 1)
        for n in (1, 2, 64, 192):
            assert 1 <= plan.splits(n, n_out) <= 38
