// q8_kv_plan.h -- the arithmetic of the page plans, for the kernels and for tests on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define Q8_HD __host__ __device__ __forceinline__
#else
#define Q8_HD inline
#endif

namespace q8 {

Q8_HD int pages_of(int64_t tokens, uint32_t shift) { return (int)((tokens + (1 << shift) - 1) >> shift); }

// New pages of a row that grows from n to n + more tokens (both >= 0); -1: its entries do not hold them, or the
// pool (n_pages) does not.
Q8_HD int new_pages(int n, int more, uint32_t max_pages, uint32_t shift, uint32_t n_pages) {
    const int64_t grown = (int64_t)n + more;
    if (grown > ((int64_t)max_pages << shift)) return -1;
    const int need = pages_of(grown, shift) - pages_of(n, shift);
    return (uint32_t)need > n_pages ? -1 : need;
}

// Sums of needs stop at `cap`, one page more than the pool has: 1024 requests of 2^24 pages do not fit 32 bits, and
// a call that needs more than the pool is refused whatever the sum.  Sums below cap are exact.  a, b <= cap <= 2^30.
Q8_HD int add_pages(int a, int b, int cap) { return a + b < cap ? a + b : cap; }

}  // namespace q8
