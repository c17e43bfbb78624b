"""The page plans' arithmetic on the host: csrc/q8_kv_plan.h, compiled as plain C++."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "q8_quantized_matmul_gb300", "csrc")
SOURCE = """
#include "q8_kv_plan.h"
extern "C" int total_of(const int *v, int n, int cap) {
    int s = 0;
    for (int i = 0; i < n; ++i) s = q8::add_pages(s, v[i], cap);
    return s;
}
// as the kernel adds: 32 values of a warp in doubling steps, then the warps
extern "C" int total_in_steps(const int *v, int n, int cap) {
    int total = 0;
    for (int w = 0; w < n; w += 32) {
        int x[32];
        for (int i = 0; i < 32; ++i) x[i] = w + i < n ? v[w + i] : 0;
        for (int o = 1; o < 32; o <<= 1)
            for (int i = 31; i >= o; --i) x[i] = q8::add_pages(x[i], x[i - o], cap);
        total = q8::add_pages(total, x[31], cap);
    }
    return total;
}
extern "C" int new_pages(int n, int more, unsigned max_pages, unsigned shift, unsigned n_pages) {
    return q8::new_pages(n, more, max_pages, shift, n_pages);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    so = str(d / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error", "-I", CSRC,
                    str(d / "plan.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


@pytest.mark.parametrize("n,each", [(128, 1 << 24), (256, 1 << 24), (1024, 1 << 21), (1024, 1 << 24), (2048, 1 << 21)])
@pytest.mark.parametrize("n_pages", [1, 1000, (1 << 24) - 1, 1 << 24])
def test_sums_beyond_32_bits_stay_above_the_pool(plan, n, each, n_pages):
    """Needs that sum to 2^31 and more: the total must not come out as something the pool holds."""
    v = np.full(n, min(each, n_pages + 1), np.int32)
    cap = n_pages + 1
    for f in (plan.total_of, plan.total_in_steps):
        total = f(v.ctypes.data_as(ctypes.c_void_p), n, cap)
        assert total == min(int(v.astype(np.int64).sum()), cap)


def test_sums_within_the_pool_are_exact(plan):
    v = np.random.default_rng(0).integers(0, 9, 5000).astype(np.int32)
    for cap in (int(v.sum()) + 1, 1 << 24):
        for f in (plan.total_of, plan.total_in_steps):
            assert f(v.ctypes.data_as(ctypes.c_void_p), len(v), cap) == v.sum()


def test_new_pages(plan):
    f = plan.new_pages
    assert f(0, 0, 4, 4, 9) == 0 and f(0, 1, 4, 4, 9) == 1 and f(16, 1, 4, 4, 9) == 1 and f(15, 1, 4, 4, 9) == 0
    assert f(0, 64, 4, 4, 9) == 4 and f(0, 65, 4, 4, 9) == -1                  # the row's entries
    assert f(0, 64, 4, 4, 3) == -1 and f(0, 48, 4, 4, 3) == 3                  # the pool
    assert f(1 << 28, (1 << 31) - 1, 1 << 24, 4, 1 << 24) == -1               # no sum in 32 bits
    assert f(0, 1 << 28, 1 << 24, 4, 1 << 24) == 1 << 24
