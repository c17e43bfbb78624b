// q8_attn_decode.cuh -- what the decode attention kernels share.
#pragma once

#include "q8_attn.cuh"
#include "q8_kv.h"

namespace q8 {

struct Seq {
    int lo, hi;          // visible positions [lo, hi)
    int start;           // lo rounded down to a multiple of `align`: the first staged position
    int tiles;
};

// Tiles of tt positions from a multiple of align on.
__device__ __forceinline__ Seq seq_of(int tt, int align, const AttnDecodeParams &p, uint32_t s, bool raise) {
    const int64_t most = (int64_t)p.max_pages << p.c.page_shift;
    int64_t n = p.lens[s];
    if (n < 0 || n > most) {
        if (raise) raise_error(p.err, DEV_ERANGE);
        n = n < 0 ? 0 : most;
    }
    Seq q;
    q.hi = (int)n;
    q.lo = p.window && n > p.window ? (int)(n - p.window) : 0;
    q.start = q.lo & ~(align - 1);
    q.tiles = (q.hi - q.start + tt - 1) / tt;
    return q;
}

// Final values of one output chunk (8 dims of a head).
__device__ __forceinline__ void finish8(const AttnDecodeParams &p, uint32_t s, uint32_t head, int d0, float m, float l,
                                        float (&o)[8], bool active) {
    float lse;
    const float f = softmax_finish(m, l, p.sinks != nullptr, p.sinks && active ? p.sinks[head] * 1.4426950408889634f : 0.0f,
                                   lse);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = f == 0.0f ? 0.0f : o[e] * f;
    const uint64_t row = (uint64_t)s * p.n_heads + head;
    store_out8(p.out, p.out_type, row * p.c.dim + d0, o, active);
    if (active && p.lse && d0 == 0) p.lse[row] = lse;
}

}  // namespace q8
