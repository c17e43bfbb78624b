// q8_attn.cuh -- device helpers shared by the attention and cache kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/q8.h"
#include "q8_common.cuh"
#include "q8_quant.cuh"

namespace q8 {

// mbar_wait for waits that mostly end at once or after a few tries: the clock is read only once a wait lasts, for a
// read takes longer than they do.  The matrix kernels, whose waits are long, keep mbar_wait (with this one their
// 4-token calls took 9.5 us instead of 8.6).
__device__ __forceinline__ bool tile_wait(uint64_t *bar, uint32_t parity, int *err, volatile int *abort,
                                          uint64_t limit_ns = WAIT_LIMIT_NS) {
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 255u) == 31u) {
            if (abort && *abort) return false;
            const uint64_t t = global_timer_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > limit_ns) {
                raise_error(err, DEV_ETIMEOUT);
                if (abort) *abort = 1;
                return false;
            }
        }
    }
}

// Programmatic launches: the wait for the kernel before this one.  (Leave for the next kernel to start early,
// griddepcontrol.launch_dependents, measured slower or no faster in every attention kernel: its waiting CTAs take
// slots and cache from this one.  64x512 decode 32 -> 36 us, 8192-token prompt 390 -> 408, small calls the same, when those took 32 and 390.)
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// 2^x on the special-function unit (relative error about 2^-22; 2^-inf = 0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The power of two that a row's weights are counted in: with the largest score (log2 units) at x they are 2^(z - r),
// r = x - UP.  In fp16 a weight below 2^-14 loses bits and one below 2^-25 is nothing, so the largest is put at 2^UP:
// one key far ahead of 60 000 others would else take the little that each of these has.  Of scores beyond 2^20 (steps of
// 1/8) x itself: the rounding of z - r could take 2^UP past the largest fp16 number.
template <int UP> __device__ __forceinline__ float weight_ref(float x) {
    if constexpr (UP == 0) return x;
    return fabsf(x) < 1048576.0f ? x - (float)UP : x;
}
// UP of the kernels whose weights pass the largest one by up to 2^8 before they rescale.
template <bool BF16> constexpr int LAZY_UP = BF16 ? 0 : 7;

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Packed fp32 pairs.
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split2(float &a, float &b, uint64_t v) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Two fp32 rounded to nearest even and packed, lo in the low half.
template <bool BF16> __device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    uint32_t r;
    if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// D (16 x 8, fp32) += A (16 x 16) * B (16 x 8), fp16 or bf16 operands.
template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// 16 bytes global -> shared, asynchronous; zeros when !valid (src is then not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Four int8 as fp32: 2^23 + (q + 128) is put together from its bytes (conversions run at a quarter of the rate).
__device__ __forceinline__ void quants4(float (&v)[4], uint32_t q) {
    q ^= 0x80808080u;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(__byte_perm(q, 0x4b000000u, 0x7440 + e)) - 8388736.0f;
}

__device__ __forceinline__ void load8s(float (&y)[8], const float *p) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    y[0] = a.x; y[1] = a.y; y[2] = a.z; y[3] = a.w;
    y[4] = b.x; y[5] = b.y; y[6] = b.z; y[7] = b.w;
}

// Softmax row totals -> factor of the unnormalised output, and the log of the denominator.
// The row's terms are sums of 2^(z - m): l of them plus, with a sink logit (log2 units), its own.
__device__ __forceinline__ float softmax_finish(float m, float l, bool has_sink, float sink, float &lse) {
    float f = 1.0f, total = l, mt = m;
    if (has_sink) {
        mt = fmaxf(m, sink);
        if (mt == -INFINITY) mt = 0.0f;                // both empty: total stays 0
        f = m == -INFINITY ? 0.0f : ex2(m - mt);
        total = l * f + ex2(sink == mt ? 0.0f : sink - mt);   // a sink of +inf takes all the weight: inf - inf is no number
    }
    lse = total == 0.0f ? -INFINITY : (mt + log2f(total)) * 0.6931471805599453f;
    return total == 0.0f ? 0.0f : f / total;
}

// Eight consecutive output values (row-major index i0, a multiple of 8) in the output's type.
// Q8_0: lanes 4i..4i+3 hold one 32-value block and every lane of the warp takes part
// (active false: nothing is stored).
__device__ __forceinline__ void store_out8(void *out, int type, uint64_t i0, const float (&y)[8], bool active) {
    if (type == Q8_TYPE_Q8_0) {
        const QuantBlock b = quantize8(y);
        if (!active) return;
        uint8_t *blk = static_cast<uint8_t *>(out) + i0 / QK * QB;
        uint16_t *dst = reinterpret_cast<uint16_t *>(blk + 2 + i0 % QK);
        dst[0] = (uint16_t)b.lo;
        dst[1] = (uint16_t)(b.lo >> 16);
        dst[2] = (uint16_t)b.hi;
        dst[3] = (uint16_t)(b.hi >> 16);
        if (i0 % QK == 0) *reinterpret_cast<uint16_t *>(blk) = b.dh;
        return;
    }
    if (!active) return;
    if (type == Q8_TYPE_F32) {
        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(out) + i0);
        dst[0] = make_float4(y[0], y[1], y[2], y[3]);
        dst[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else if (type == Q8_TYPE_BF16) {
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + i0) =
            make_uint4(pack16<true>(y[0], y[1]), pack16<true>(y[2], y[3]), pack16<true>(y[4], y[5]),
                       pack16<true>(y[6], y[7]));
    } else {
        *reinterpret_cast<uint4 *>(static_cast<__half *>(out) + i0) =
            make_uint4(pack16<false>(y[0], y[1]), pack16<false>(y[2], y[3]), pack16<false>(y[4], y[5]),
                       pack16<false>(y[6], y[7]));
    }
}

}  // namespace q8
