// q8_residual.cu -- the residual path between two blocks in one pass over its rows:
//   u  = y  or  (y r(y)) gamma_post,   h' = residual_scale h + gate u,   n = (h' r(h')) gamma_next,
//   r(x) = 1 / sqrt(S / dim + eps),  S = sum x^2.
// Every product, sum, quotient and root is rounded to fp32 on its own.  S is carried in two fp32 words (each square
// with its rounding error, each addition with its own), so that its one rounding to fp32 hardly ever depends on the
// order of the sum (error below 2^-37, 2^-46 as a rule, against the 2^-24 of the rounding; |x| >= 2^-51): Q8_0 bytes can be
// told from the definition alone but in one row of some 2^20.
// In packed pairs that is 5 instructions a value for each norm.  4096 rows of 4096, fp32, gated, both norms, Q8_0 out: 53.5 us, 4.1 TB/s
// (bound by the joins, two a row with two barriers each: barrier 7.2 cycles an issue, issue 50 % busy, DRAM 41 %; a
// ring of asynchronous copies 73 us, two or four chunks a thread 55 to 58).
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

// The sums of the even and of the odd values' squares: twelve instructions for two values, of a thread's first two four.  The products are taken one by
// one: a packed product that a packed sum uses is made one fused operation with it, whatever the rounding both ask for.
struct Squares {
    uint64_t hi = 0, lo = 0;
    __device__ __forceinline__ void add_square(uint64_t x, bool first) {
        float x0, x1;
        split2(x0, x1, x);
        const float p0 = __fmul_rn(x0, x0), p1 = __fmul_rn(x1, x1);
        const uint64_t p = pair2(p0, p1), e = pair2(__fmaf_rn(x0, x0, -p0), __fmaf_rn(x1, x1, -p1));      // x^2 = p + e
        if (first) {
            hi = p;
            lo = e;
            return;
        }
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

__device__ __forceinline__ float inverse_rms(float total, float dim, float eps) {
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(total, dim), eps)));
}

__device__ __forceinline__ Sum2 lane_sum(Sum2 s, int from) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        if (o <= from) s = add(s, {__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
    return s;
}

// r of the whole CTA's values on every thread.  part: words that no other call of the row uses.  ONE_WARP: one warp joins every
// thread's sums and takes the root (a longer chain, but 100 instructions less in every other warp); else each warp joins its
// own, and then all of them for itself.
template <int MAXT, bool ONE_WARP> struct Part {
    Sum2 sums[ONE_WARP ? MAXT : 32];
    float r;
};
template <int MAXT, bool ONE_WARP>
__device__ __forceinline__ float cta_inverse_rms(const Squares &q, Part<MAXT, ONE_WARP> &part, float dim, float eps) {
    Sum2 s = q.both();
    const int lane = threadIdx.x & 31, warps = (int)(blockDim.x >> 5);
    if constexpr (ONE_WARP) {
        part.sums[threadIdx.x] = s;
        __syncthreads();
        if (threadIdx.x < 32) {
            for (int w = 1; w < warps; ++w) s = add(s, part.sums[w * 32 + lane]);
            s = lane_sum(s, 16);
            if (lane == 0) part.r = inverse_rms(isinf(s.hi) ? s.hi : __fadd_rn(s.hi, s.lo), dim, eps);
        }
        __syncthreads();
        return part.r;
    } else {
        s = lane_sum(s, 16);
        if (lane == 0) part.sums[threadIdx.x >> 5] = s;
        __syncthreads();
        s = lane < warps ? part.sums[lane] : Sum2{0.0f, 0.0f};
        s = lane_sum(s, warps > 16 ? 16 : warps > 8 ? 8 : warps > 4 ? 4 : warps > 2 ? 2 : warps > 1 ? 1 : 0);
        s.hi = __shfl_sync(0xffffffffu, s.hi, 0);
        s.lo = __shfl_sync(0xffffffffu, s.lo, 0);
        return inverse_rms(isinf(s.hi) ? s.hi : __fadd_rn(s.hi, s.lo), dim, eps);
    }
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

__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The quantiser (see quantize8: the same bytes) of eight values a lane, four lanes a block, in packed pairs: k, the whole number
// next to x (1 / d) with an approximate 1 / d, is roundf(x / d) where the two differ by less than 0.4999 (their errors reach
// 3 2^-23 128 < 5e-5); a lane with one that does not (or with a d of no reciprocal: the difference is then no number) divides.
__device__ __forceinline__ void quantize8_pairs(const uint64_t (&x)[4], uint32_t &lo, uint32_t &hi, uint16_t &dh) {
    float v[8];
    unpack(v, x);
    float amax = fmaxf(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))),
                       fmaxf(fmaxf(fabsf(v[4]), fabsf(v[5])), fmaxf(fabsf(v[6]), fabsf(v[7]))));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const float d = __fdiv_rn(amax, 127.0f);
    float rd;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rd) : "f"(d));
    const uint64_t rd2 = pair2(rd, rd), magic = pair2(ROUND_MAGIC, ROUND_MAGIC);
    uint32_t t[8];
    float off = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint64_t sm = fma2(x[e], rd2, magic), r = fma2(x[e], rd2, sub2(magic, sm));
        float a, b, ra, rb;
        split2(a, b, sm);
        split2(ra, rb, r);
        t[2 * e] = __float_as_uint(a);
        t[2 * e + 1] = __float_as_uint(b);
        off = max_nan(off, max_nan(fabsf(ra), fabsf(rb)));
    }
    lo = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
    hi = __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410);
    dh = __half_as_ushort(__float2half_rn(d));
    if (!(off < 0.4999f)) {
        lo = hi = 0;
        if (d != 0.0f) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lo |= (uint32_t)(uint8_t)(int8_t)(int)roundf(__fdiv_rn(v[e], d)) << (8 * e);
                hi |= (uint32_t)(uint8_t)(int8_t)(int)roundf(__fdiv_rn(v[4 + e], d)) << (8 * e);
            }
        }
    }
}

// A warp's 32 chunks of a row as Q8_0 (272 bytes; less at the row's end), through shared memory: written by its lanes, 34 bytes apart
// and two at a time, a row took four times the sectors.
__device__ __forceinline__ void store_q8_warp(uint8_t *dst, uint8_t *stage, const uint64_t (&n)[4], uint32_t live_chunks) {
    const uint32_t lane = threadIdx.x & 31u;
    uint32_t lo, hi;
    uint16_t dh;
    quantize8_pairs(n, lo, hi, dh);
    uint16_t *at = reinterpret_cast<uint16_t *>(stage + lane / 4 * QB + 2 + lane % 4 * 8);
    at[0] = (uint16_t)lo;
    at[1] = (uint16_t)(lo >> 16);
    at[2] = (uint16_t)hi;
    at[3] = (uint16_t)(hi >> 16);
    if (lane % 4 == 0) at[-1] = dh;
    __syncwarp();
    const uint32_t bytes = live_chunks / 4 * QB;
    if (bytes == 272 && (reinterpret_cast<uintptr_t>(dst) & 15u) == 0) {
        if (lane < 17) reinterpret_cast<uint4 *>(dst)[lane] = reinterpret_cast<const uint4 *>(stage)[lane];
    } else {
        for (uint32_t i = lane; i < bytes / 2; i += 32) reinterpret_cast<uint16_t *>(dst)[i] = reinterpret_cast<const uint16_t *>(stage)[i];
    }
    __syncwarp();
}

// One CTA a row at a time; a thread has chunks of 8 values t, t + T, ..., NS of them.  MANY: for many rows a CTA: the next row is
// loaded while this one is worked on, one warp takes the roots.
template <int NS, int MAXT, int MINB, bool MANY, bool HWIDE, bool YWIDE>
__global__ void __launch_bounds__(MAXT, MINB) k_residual_norm(const ResidualNormParams p, int h_type, int y_type) {
    __shared__ __align__(16) uint8_t stages[MAXT / 32][272];
    __shared__ Part<MAXT, MANY> part[2];
    const uint32_t chunks = p.dim / 8, t = threadIdx.x, T = blockDim.x;
    const float dim = (float)p.dim;
    const bool hbf = h_type == Q8_TYPE_BF16, ybf = y_type == Q8_TYPE_BF16, whole = p.whole;
    const uint32_t row_bytes = p.dim / QK * QB;
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
    if (MANY) load_row(blockIdx.x);
    for (uint64_t row = blockIdx.x; row < p.n_tok; row += gridDim.x) {
        const float *gate = p.gate ? p.gate + row * p.gate_stride : nullptr;
        if (!MANY) load_row(row);
        float ry = 1.0f;
        if (p.post) {
            Squares acc;
#pragma unroll
            for (int s = 0; s < NS; ++s)
                if (t + s * T < chunks) {
                    uint64_t v[4];
                    values<YWIDE>(v, yraw[s], ybf);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc.add_square(v[e], s == 0 && e == 0);
                }
            ry = cta_inverse_rms(acc, part[0], dim, p.eps);
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
                for (int e = 0; e < 4; ++e) u[e] = mul2(u[e], ry2);
                if (p.gamma_post) {
                    load_pairs(g, p.gamma_post + c * 8, whole);
#pragma unroll
                    for (int e = 0; e < 4; ++e) u[e] = mul2(u[e], g[e]);
                }
            }
            if (gate) {
                load_pairs(g, gate + c * 8, whole);
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] = mul2(g[e], u[e]);
            }
            float h[8], v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) hv[s][e] = mul2(scale2, hv[s][e]);
            unpack(h, hv[s]);
            unpack(v, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = __fadd_rn(h[e], v[e]);   // one by one: see Squares
#pragma unroll
            for (int e = 0; e < 4; ++e) hv[s][e] = pair2(h[2 * e], h[2 * e + 1]);
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
            for (int e = 0; e < 4; ++e) acc.add_square(hv[s][e], s == 0 && e == 0);
        }
        if (MANY && row + gridDim.x < p.n_tok) load_row(row + gridDim.x);
        if (!p.n_out) {
            if (p.post) __syncthreads();   // part[0] of the next row
            continue;
        }
        const float rh = cta_inverse_rms(acc, part[1], dim, p.eps);
        const uint64_t rh2 = pair2(rh, rh);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const uint32_t c = t + s * T;
            if ((c & ~31u) >= chunks) continue;      // whole warps: the quantiser shuffles
            uint64_t g[4];
            if (c < chunks) {
#pragma unroll
                for (int e = 0; e < 4; ++e) hv[s][e] = mul2(hv[s][e], rh2);
                if (p.gamma_next) {
                    load_pairs(g, p.gamma_next + c * 8, whole);
#pragma unroll
                    for (int e = 0; e < 4; ++e) hv[s][e] = mul2(hv[s][e], g[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) hv[s][e] = 0;
            }
            if (p.n_type == Q8_TYPE_Q8_0) {
                const uint32_t c0 = c & ~31u;
                store_q8_warp(static_cast<uint8_t *>(p.n_out) + row * row_bytes + (uint64_t)c0 / 4 * QB, stages[t / 32], hv[s], min(32u, chunks - c0));
            } else {
                float n[8];
                unpack(n, hv[s]);
                store8(p.n_out, p.n_type, row * p.dim + (uint64_t)c * 8, n, c < chunks, whole);
            }
        }
        // part[0] is written again after part[1]'s barriers, part[1] after part[0]'s (none without the first norm)
        if (!p.post) __syncthreads();
    }
}

template <int NS, int MAXT, int MINB, bool MANY, bool HWIDE, bool YWIDE>
cudaError_t launch_rows(const ResidualNormParams &p, int h_type, int y_type, int num_sms, cudaStream_t st) {
    const auto kernel = k_residual_norm<NS, MAXT, MINB, MANY, HWIDE, YWIDE>;
    cudaLaunchConfig_t cfg = {};
    const unsigned threads = (p.dim / 8 + NS - 1) / NS + 31 & ~31u;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaSuccess;
    int fit = 1;
    if (p.n_tok > (uint64_t)num_sms) {
        if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, (int)threads, 0)) != cudaSuccess) return e;
        if (fit < 1) fit = 1;
    }
    const uint64_t ctas = (uint64_t)num_sms * fit;
    cfg.gridDim = dim3((unsigned)(p.n_tok < ctas ? p.n_tok : ctas));
    e = cudaLaunchKernelEx(&cfg, kernel, p, h_type, y_type);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// Few rows: as many threads a row as it has chunks, the shortest chain.  Many rows: of up to 4096 values the same, each CTA with its next
// row on the way (4096 x 4096 with both norms: 53.5 us; 608 rows 8.8, without the row ahead 9.4, but 304 rows 5.3 without); of
// more, 32 values a thread (4096 x 8192: 110 us against 140 with 8 or with a row ahead).  Above 16384 values 64 registers a thread do not
// hold them, and 232 to 744 bytes a thread are spilled (2048 rows of 16384: 139 us, of 16416: 228, of 32768: 375).
template <bool HWIDE, bool YWIDE>
cudaError_t launch_typed(const ResidualNormParams &p, int h_type, int y_type, int num_sms, cudaStream_t st) {
    const uint32_t chunks = p.dim / 8;
    const bool few = p.n_tok <= (uint64_t)(2 * num_sms);
    if (chunks <= 512)
        return few ? launch_rows<1, 512, 2, false, HWIDE, YWIDE>(p, h_type, y_type, num_sms, st)
                   : launch_rows<1, 512, 2, true, HWIDE, YWIDE>(p, h_type, y_type, num_sms, st);
    if (chunks <= 1024)
        return few ? launch_rows<1, 1024, 1, false, HWIDE, YWIDE>(p, h_type, y_type, num_sms, st)
                   : launch_rows<4, 256, 2, false, HWIDE, YWIDE>(p, h_type, y_type, num_sms, st);
    if (chunks <= 2048) return launch_rows<4, 512, 1, false, HWIDE, YWIDE>(p, h_type, y_type, num_sms, st);
    return launch_rows<4, 1024, 1, false, HWIDE, YWIDE>(p, h_type, y_type, num_sms, st);
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
