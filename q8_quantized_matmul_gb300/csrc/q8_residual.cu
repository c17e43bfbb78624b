// q8_residual.cu -- the residual path between two blocks in one pass over its rows:
//   u  = y  or  (y r(y)) gamma_post,   h' = residual_scale h + gate u,   n = (h' r(h')) gamma_next,
//   r(x) = 1 / sqrt(S / dim + eps),  S = sum x^2.
// Every product, sum, quotient and root is rounded to fp32 on its own.  S is carried in two fp32 words (each square
// with its rounding error, each addition with its own), so that its one rounding to fp32 hardly ever depends on the
// order of the sum (2^-44 against the 2^-24 of the rounding): Q8_0 bytes can be told from the definition alone.
// In packed pairs that is 6 instructions a value for each norm, which the memory hides.
#include "q8_attn.cuh"
#include "q8_kv.h"
#include "q8_layer.h"

namespace q8 {
namespace {

// Packed fp32 pairs, each half rounded on its own.
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A sum in two words, hi + lo.
struct Sum2 {
    float hi, lo;
};

// s + t, the rounding error of the high words kept (Knuth's exact addition).
__device__ __forceinline__ Sum2 add(Sum2 s, Sum2 t) {
    const float hi = __fadd_rn(s.hi, t.hi), b = __fsub_rn(hi, s.hi);
    const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(hi, b)), __fsub_rn(t.hi, b));
    return {hi, __fadd_rn(__fadd_rn(s.lo, t.lo), e)};
}

// The products of two pairs, each on its own: a packed product whose only use is a packed sum is made one fused
// operation with it, whatever the rounding that both ask for.
__device__ __forceinline__ uint64_t mul2_alone(uint64_t a, uint64_t b) {
    float a0, a1, b0, b1;
    split2(a0, a1, a);
    split2(b0, b1, b);
    return pair2(__fmul_rn(a0, b0), __fmul_rn(a1, b1));
}

// The sums of the even and of the odd values' squares: twelve instructions for two values.
struct Squares {
    uint64_t hi = 0, lo = 0;
    __device__ __forceinline__ void operator+=(uint64_t x) {
        float x0, x1;
        split2(x0, x1, x);
        const float p0 = __fmul_rn(x0, x0), p1 = __fmul_rn(x1, x1);
        const uint64_t p = pair2(p0, p1), e = pair2(__fmaf_rn(x0, x0, -p0), __fmaf_rn(x1, x1, -p1));      // x^2 = p + e
        const uint64_t s = add2(hi, p), b = sub2(s, hi), r = add2(sub2(hi, sub2(s, b)), sub2(p, b));
        hi = s;
        lo = add2(lo, add2(r, e));
    }
    __device__ __forceinline__ Sum2 both() const {
        Sum2 a, b;
        split2(a.hi, b.hi, hi);
        split2(a.lo, b.lo, lo);
        return add(a, b);
    }
};

// The whole CTA's sum, rounded to fp32, on every thread.  part: 32 words that no other call of the row uses.
__device__ __forceinline__ float cta_sum(const Squares &q, Sum2 *part) {
    Sum2 s = q.both();
#pragma unroll
    for (int o = 16; o; o >>= 1)
        s = add(s, {__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
    const int lane = threadIdx.x & 31, warps = (int)(blockDim.x >> 5);
    if (lane == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = lane < warps ? part[lane] : Sum2{0.0f, 0.0f};
#pragma unroll
    for (int o = 16; o; o >>= 1)
        if (o < warps) s = add(s, {__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
    s.hi = __shfl_sync(0xffffffffu, s.hi, 0);
    s.lo = __shfl_sync(0xffffffffu, s.lo, 0);
    return isinf(s.hi) ? s.hi : __fadd_rn(s.hi, s.lo);
}

__device__ __forceinline__ float inverse_rms(float total, float dim, float eps) {
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(total, dim), eps)));
}

// 32 bytes of a row at once where it starts on such a boundary, else 16 at a time.
__device__ __forceinline__ void load32(uint32_t *w, const void *p, bool whole) {
    if (whole) {
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
        const uint4 a = static_cast<const uint4 *>(p)[0], b = static_cast<const uint4 *>(p)[1];
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
}

// Eight values as they lie in memory.
template <bool WIDE> struct Raw8 {
    uint32_t w[WIDE ? 8 : 4];
};

template <bool WIDE> __device__ __forceinline__ void load_raw(Raw8<WIDE> &r, const uint8_t *row, uint32_t chunk, bool whole) {
    if constexpr (WIDE) {
        load32(r.w, row + (uint64_t)chunk * 32, whole);
    } else {
        const uint4 v = *reinterpret_cast<const uint4 *>(row + (uint64_t)chunk * 16);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    }
}

// The same as four fp32 pairs.
template <bool WIDE> __device__ __forceinline__ void values(uint64_t (&v)[4], const Raw8<WIDE> &r, bool bf16) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (WIDE) v[e] = pair2(__uint_as_float(r.w[2 * e]), __uint_as_float(r.w[2 * e + 1]));
        else if (bf16) v[e] = pair2(__uint_as_float(r.w[e] << 16), __uint_as_float(r.w[e] & 0xffff0000u));
        else v[e] = pair2(half_bits_to_float((uint16_t)r.w[e]), half_bits_to_float((uint16_t)(r.w[e] >> 16)));
    }
}

__device__ __forceinline__ void load_pairs(uint64_t (&v)[4], const float *p, bool whole) {
    Raw8<true> r;
    load32(r.w, p, whole);
    values<true>(v, r, false);
}

__device__ __forceinline__ void unpack(float (&y)[8], const uint64_t (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(y[2 * e], y[2 * e + 1], v[e]);
}

// store_out8 with fp32 written 32 bytes at once where the rows allow it.
__device__ __forceinline__ void store8(void *out, int type, uint64_t i0, const float (&y)[8], bool active, bool whole) {
    if (type == Q8_TYPE_F32 && whole) {
        if (active)
            asm volatile("st.global.v8.f32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]),
                         "f"(y[5]), "f"(y[6]), "f"(y[7]), "l"(static_cast<float *>(out) + i0)
                         : "memory");
        return;
    }
    store_out8(out, type, i0, y, active);
}

// One CTA a row at a time; a thread has chunks of 8 values t, t + T, ..., NS of them.  AHEAD: the next row is loaded while
// this one is worked on.
template <int NS, int MAXT, int MINB, bool AHEAD, bool HWIDE, bool YWIDE>
__global__ void __launch_bounds__(MAXT, MINB) k_residual_norm(const ResidualNormParams p, int h_type, int y_type) {
    __shared__ Sum2 part[2][32];
    const uint32_t chunks = p.dim / 8, t = threadIdx.x, T = blockDim.x;
    const float dim = (float)p.dim;
    const bool hbf = h_type == Q8_TYPE_BF16, ybf = y_type == Q8_TYPE_BF16, whole = p.whole;
    const uint64_t scale2 = pair2(p.residual_scale, p.residual_scale);
    Raw8<YWIDE> yraw[NS];
    Raw8<HWIDE> hraw[NS];
    const auto load_row = [&](uint64_t row) {
        const uint8_t *yr = static_cast<const uint8_t *>(p.y) + row * p.y_stride * (YWIDE ? 4 : 2);
        const uint8_t *hr = static_cast<const uint8_t *>(p.h) + row * p.h_stride * (HWIDE ? 4 : 2);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const uint32_t c = t + s * T;
            if (c < chunks) {
                load_raw<YWIDE>(yraw[s], yr, c, whole);
                load_raw<HWIDE>(hraw[s], hr, c, whole);
            }
        }
    };
    grid_dep_wait();
    if (AHEAD) load_row(blockIdx.x);
    for (uint64_t row = blockIdx.x; row < p.n_tok; row += gridDim.x) {
        const float *gate = p.gate ? p.gate + row * p.gate_stride : nullptr;
        if (!AHEAD) load_row(row);
        float ry = 1.0f;
        if (p.post) {
            Squares acc;
#pragma unroll
            for (int s = 0; s < NS; ++s)
                if (t + s * T < chunks) {
                    uint64_t v[4];
                    values<YWIDE>(v, yraw[s], ybf);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc += v[e];
                }
            ry = inverse_rms(cta_sum(acc, part[0]), dim, p.eps);
        }
        const uint64_t ry2 = pair2(ry, ry);
        uint64_t hv[NS][4];
        Squares acc;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const uint32_t c = t + s * T;
            if (c >= chunks) continue;
            uint64_t u[4], g[4];
            values<YWIDE>(u, yraw[s], ybf);
            values<HWIDE>(hv[s], hraw[s], hbf);
            if (p.post) {
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] = mul2_alone(u[e], ry2);
                if (p.gamma_post) {
                    load_pairs(g, p.gamma_post + c * 8, whole);
#pragma unroll
                    for (int e = 0; e < 4; ++e) u[e] = mul2_alone(u[e], g[e]);
                }
            }
            if (gate) {
                load_pairs(g, gate + c * 8, whole);
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] = mul2_alone(g[e], u[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) hv[s][e] = add2(mul2_alone(scale2, hv[s][e]), u[e]);
            float h[8];
            unpack(h, hv[s]);
            if constexpr (!HWIDE) {   // the next norm is of the stored value
                Raw8<false> r;
#pragma unroll
                for (int e = 0; e < 4; ++e) r.w[e] = hbf ? pack16<true>(h[2 * e], h[2 * e + 1]) : pack16<false>(h[2 * e], h[2 * e + 1]);
                values<false>(hv[s], r, hbf);
                if (p.h_out)
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.h_out) + row * p.h_out_stride + c * 8) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
            } else if (p.h_out) {
                store8(p.h_out, Q8_TYPE_F32, row * p.h_out_stride + c * 8, h, true, whole);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc += hv[s][e];
        }
        if (AHEAD && row + gridDim.x < p.n_tok) load_row(row + gridDim.x);
        if (!p.n_out) {
            if (p.post) __syncthreads();   // part[0] of the next row
            continue;
        }
        const float rh = inverse_rms(cta_sum(acc, part[1]), dim, p.eps);
        const uint64_t rh2 = pair2(rh, rh);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const uint32_t c = t + s * T;
            if ((c & ~31u) >= chunks) continue;      // whole warps: the quantiser shuffles
            uint64_t g[4];
            float n[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (c < chunks) {
#pragma unroll
                for (int e = 0; e < 4; ++e) hv[s][e] = mul2(hv[s][e], rh2);
                if (p.gamma_next) {
                    load_pairs(g, p.gamma_next + c * 8, whole);
#pragma unroll
                    for (int e = 0; e < 4; ++e) hv[s][e] = mul2(hv[s][e], g[e]);
                }
                unpack(n, hv[s]);
            }
            store8(p.n_out, p.n_type, row * p.dim + (uint64_t)c * 8, n, c < chunks, whole);
        }
        // part[0] is written again after part[1]'s barrier, part[1] after part[0]'s (none without the first norm)
        if (!p.post) __syncthreads();
    }
}

template <class K>
cudaError_t launch_rows(K kernel, const ResidualNormParams &p, int h_type, int y_type, int threads, int ctas, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.n_tok < (uint64_t)ctas ? p.n_tok : (uint64_t)ctas));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, h_type, y_type);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

template <bool HWIDE, bool YWIDE>
cudaError_t launch_typed(const ResidualNormParams &p, int h_type, int y_type, int num_sms, cudaStream_t st) {
    const uint32_t chunks = p.dim / 8;
    const auto threads = [&](int ns) { return (int)((chunks + ns - 1) / ns + 31) & ~31; };
    // CTAs that fill the SMs: 65536 registers, 32 CTAs
    const auto ctas = [&](int ns, int regs) {
        const int per = 65536 / (regs * threads(ns));
        return num_sms * (per > 32 ? 32 : per < 1 ? 1 : per);
    };
    if (chunks <= 512)
        return launch_rows(k_residual_norm<1, 512, 2, true, HWIDE, YWIDE>, p, h_type, y_type, threads(1), ctas(1, 64), st);
    if (chunks <= 1024)
        return launch_rows(k_residual_norm<2, 512, 1, true, HWIDE, YWIDE>, p, h_type, y_type, threads(2), ctas(2, 128), st);
    if (chunks <= 2048)
        return launch_rows(k_residual_norm<4, 512, 1, false, HWIDE, YWIDE>, p, h_type, y_type, threads(4), ctas(4, 128), st);
    return launch_rows(k_residual_norm<4, 1024, 1, false, HWIDE, YWIDE>, p, h_type, y_type, threads(4), ctas(4, 64), st);
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormParams &q, int h_type, int y_type, int num_sms, cudaStream_t st) {
    const bool hw = h_type == Q8_TYPE_F32, yw = y_type == Q8_TYPE_F32;
    ResidualNormParams p = q;
    // fp32 rows that all start on 32-byte boundaries
    uint64_t bits = (uint64_t)(uintptr_t)p.gamma_post | (uint64_t)(uintptr_t)p.gamma_next | (uint64_t)(uintptr_t)p.gate | p.gate_stride * 4;
    if (hw) bits |= (uint64_t)(uintptr_t)p.h | (uint64_t)(uintptr_t)p.h_out | p.h_stride * 4 | p.h_out_stride * 4;
    if (yw) bits |= (uint64_t)(uintptr_t)p.y | p.y_stride * 4;
    if (p.n_type == Q8_TYPE_F32) bits |= (uint64_t)(uintptr_t)p.n_out;
    p.whole = (bits & 31u) == 0;
    if (hw) return yw ? launch_typed<true, true>(p, h_type, y_type, num_sms, st) : launch_typed<true, false>(p, h_type, y_type, num_sms, st);
    return yw ? launch_typed<false, true>(p, h_type, y_type, num_sms, st) : launch_typed<false, false>(p, h_type, y_type, num_sms, st);
}

}  // namespace q8
