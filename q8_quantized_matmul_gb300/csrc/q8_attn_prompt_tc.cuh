// q8_attn_prompt_tc.cuh -- one thread's row of a 128 x 128 tile of scores in TMEM: what the tcgen05 prompt
// attention kernels share.
#pragma once

#include "q8_attn_prompt.cuh"
#include "q8_tcgen05.cuh"

namespace q8 {

// Row r (0 .. 127) of half i of a tile: its token within the tile (the last one for rows that hold none) and its
// head among the packed ones.
struct RowOf {
    int token, head;
    bool used;
    __device__ __forceinline__ RowOf(const AttnPromptParams &p, int i, int r) {
        const int t = r / p.pack;
        used = t < p.half;
        token = i * p.half + min(t, p.half - 1);
        head = r - t * p.pack;
    }
};

// Columns outside lo .. hi become -inf.
__device__ __forceinline__ void row_mask(uint32_t (&v)[128], int lo, int hi) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        // bits of the 32 columns from 32 b on
        const int h = hi + 1 - 32 * b, g = lo - 32 * b;
        const uint32_t below = h >= 32 ? 0xffffffffu : (h <= 0 ? 0u : (1u << h) - 1u);
        const uint32_t seen = g <= 0 ? below : (g >= 32 ? 0u : below & (0xffffffffu << g));
        if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;   // most words of an edge tile are whole
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (!(seen & (1u << c))) v[32 * b + c] = 0xff800000u;
    }
}

__device__ __forceinline__ float row_max(const uint32_t (&v)[128]) {
    float x0 = __uint_as_float(v[0]), x1 = __uint_as_float(v[1]), x2 = __uint_as_float(v[2]), x3 = __uint_as_float(v[3]);
#pragma unroll
    for (int c = 4; c < 124; c += 8) {
        x0 = max3(x0, __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
        x1 = max3(x1, __uint_as_float(v[c + 2]), __uint_as_float(v[c + 3]));
        x2 = max3(x2, __uint_as_float(v[c + 4]), __uint_as_float(v[c + 5]));
        x3 = max3(x3, __uint_as_float(v[c + 6]), __uint_as_float(v[c + 7]));
    }
    x0 = max3(x0, __uint_as_float(v[124]), __uint_as_float(v[125]));
    x1 = max3(x1, __uint_as_float(v[126]), __uint_as_float(v[127]));
    return max3(fmaxf(x0, x1), x2, x3);
}

// N columns of O times f.
template <int N> __device__ __forceinline__ void row_rescale(uint32_t tO, float f) {
#pragma unroll 1
    for (int c = 0; c < N; c += 16) {
        uint32_t o[16];
        tc_ld16(tO + c, o);
        tc_wait_ld();
        tc_regs_ready(o);
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tc_st16(tO + c, o);
    }
}

// Weights 2^(scale v - r), written as 16-bit pairs over the scores; their sum (before rounding).
template <bool BF16> __device__ __forceinline__ float row_weights(const uint32_t (&v)[128], float scale, float r, uint32_t tS) {
    const float neg = r == -INFINITY ? 0.0f : -r;
    const uint64_t scale2 = pair2(scale, scale), neg2 = pair2(neg, neg);
    uint64_t s0 = 0, s1 = 0;
#pragma unroll
    for (int b = 0; b < 128; b += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
            float a0, a1, a2, a3;
            split2(a0, a1, fma2(pair2(__uint_as_float(v[b + c]), __uint_as_float(v[b + c + 1])), scale2, neg2));
            split2(a2, a3, fma2(pair2(__uint_as_float(v[b + c + 2]), __uint_as_float(v[b + c + 3])), scale2, neg2));
            a0 = ex2(a0);
            a1 = ex2(a1);
            a2 = ex2(a2);
            a3 = ex2(a3);
            s0 = add2(s0, pair2(a0, a1));
            s1 = add2(s1, pair2(a2, a3));
            pk[c / 2] = pack16<BF16>(a0, a1);
            pk[c / 2 + 1] = pack16<BF16>(a2, a3);
        }
        tc_st16(tS + b / 2, pk);
    }
    float l0, l1;
    split2(l0, l1, add2(s0, s1));
    return l0 + l1;
}

// 32 fp32 output values of one thread's row, columns d0 ..
__device__ __forceinline__ void store_row32(const AttnPromptParams &p, uint64_t row, int d0, const float *y) {
    const uint64_t i0 = row * p.dim + d0;
    if (p.out_type == Q8_TYPE_Q8_0) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(y[i]));
        const float d = __fdiv_rn(amax, 127.0f);
        uint16_t *dst = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(p.out) + i0 / QK * QB);
        dst[0] = d != 0.0f ? __half_as_ushort(__float2half_rn(d)) : 0;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const int a = d != 0.0f ? (int)roundf(__fdiv_rn(y[2 * i], d)) : 0;
            const int b = d != 0.0f ? (int)roundf(__fdiv_rn(y[2 * i + 1], d)) : 0;
            dst[1 + i] = (uint16_t)((a & 0xff) | (b & 0xff) << 8);
        }
    } else if (p.out_type != Q8_TYPE_F32 && (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0) {
        // a thread's row leaves in whole 32-byte sectors
        const bool bf = p.out_type == Q8_TYPE_BF16;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = bf ? pack16<true>(y[2 * i], y[2 * i + 1]) : pack16<false>(y[2 * i], y[2 * i + 1]);
        uint16_t *dst = static_cast<uint16_t *>(p.out) + i0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst + 16 * i), "r"(w[8 * i]), "r"(w[8 * i + 1]),
                         "r"(w[8 * i + 2]), "r"(w[8 * i + 3]), "r"(w[8 * i + 4]), "r"(w[8 * i + 5]), "r"(w[8 * i + 6]),
                         "r"(w[8 * i + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = y[8 * i + e];
            store_out8(p.out, p.out_type, i0 + 8 * i, x, true);
        }
    }
}

// N columns of O times f as the output's dims d0 .. of `orow` (a token's head); row: the token within the tile; vp (or nullptr): the first value row
// of the sequence, at this head's first dim, when values that are not finite were taken out (prompt_restore).
template <int N, bool BF16>
__device__ __forceinline__ void row_output(const AttnPromptParams &p, const PromptTile &w, uint32_t tO, float f, bool mine,
                                           uint64_t orow, int d0, const uint16_t *vp, int row) {
#pragma unroll 1
    for (int c = 0; c < N; c += 32) {
        uint32_t o[32];
        tc_ld32(tO + c, o);
        tc_wait_ld();
        tc_regs_ready(o);
        float y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = f == 0.0f ? 0.0f : __uint_as_float(o[e]) * f;
        if (!mine) continue;
        if (vp) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
                float z[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) z[k] = y[e + k];
                prompt_restore<BF16>(p, w, vp + d0 + c + e, row, 128, z);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[e + k] = z[k];
            }
        }
        store_row32(p, orow, d0 + c, y);
    }
}

}  // namespace q8
