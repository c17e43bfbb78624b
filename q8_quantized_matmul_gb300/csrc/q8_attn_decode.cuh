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

// A head's sink in log2 units; loaded ahead of the pieces that it follows.
__device__ __forceinline__ float sink_of(const AttnDecodeParams &p, uint32_t head, bool active) {
    return p.sinks && active ? p.sinks[head] * 1.4426950408889634f : 0.0f;
}

// Final values of one output chunk (8 dims of a head).
__device__ __forceinline__ void finish8(const AttnDecodeParams &p, uint32_t s, uint32_t head, int d0, float sink, float m,
                                        float l, float (&o)[8], bool active) {
    float lse;
    const float f = softmax_finish(m, l, p.sinks != nullptr, sink, lse);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = f == 0.0f ? 0.0f : o[e] * f;
    const uint64_t row = (uint64_t)s * p.n_heads + head;
    store_out8(p.out, p.out_type, row * p.c.dim + d0, o, active);
    if (active && p.lse && d0 == 0) p.lse[row] = lse;
}

// (m, l, y) of 8 dims of a head over pieces 0 .. n - 1 in their order: src(k) the piece's values, ml(k) its maximum
// and sum.  One pass with a running maximum and eight pieces' loads in flight: the loads of a round wait for
// nothing (a pass for the maximum first costs two more trips to the L2).
template <class Src, class Ml>
__device__ __forceinline__ void join8(int n, Src src, Ml ml, float &m, float &l, float (&y)[8]) {
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = 0.0f;
    for (int k0 = 0; k0 < n; k0 += 8) {
        float4 va[8], vb[8];
        float2 x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int k = min(k0 + u, n - 1);
            x[u] = __ldcg(ml(k));
            const float4 *v = reinterpret_cast<const float4 *>(src(k));
            va[u] = __ldcg(v);
            vb[u] = __ldcg(v + 1);
        }
        float mt = m;
#pragma unroll
        for (int u = 0; u < 8; ++u) mt = fmaxf(mt, x[u].x);
        const float g = m == -INFINITY ? 0.0f : ex2(m - mt);
        m = mt;
        l *= g;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= g;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (k0 + u >= n || x[u].x == -INFINITY) continue;        // nothing seen there
            const float f = ex2(x[u].x - mt);
            l += x[u].y * f;
            y[0] += va[u].x * f;
            y[1] += va[u].y * f;
            y[2] += va[u].z * f;
            y[3] += va[u].w * f;
            y[4] += vb[u].x * f;
            y[5] += vb[u].y * f;
            y[6] += vb[u].z * f;
            y[7] += vb[u].w * f;
        }
    }
}

}  // namespace q8
