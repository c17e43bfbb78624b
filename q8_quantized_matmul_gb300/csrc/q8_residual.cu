// q8_residual.cu -- the residual path between two blocks in one pass over its rows:
//   u  = y  or  (y r(y)) gamma_post,   h' = residual_scale h + gate u,   n = (h' r(h')) gamma_next,
//   r(x) = 1 / sqrt(S / dim + eps),  S = sum x^2.
// Every product, sum, quotient and root is rounded to fp32 on its own.  S is carried in two fp32 words (each square
// with its rounding error, each addition with its own), so that its one rounding to fp32 hardly ever depends on the
// order of the sum (2^-44 against the 2^-24 of the rounding): Q8_0 bytes can be told from the definition alone.
// That is about 10 instructions a value for each norm, which the memory hides.
#include "q8_attn.cuh"
#include "q8_kv.h"
#include "q8_layer.h"

namespace q8 {
namespace {

// A sum in two words: hi + lo.
struct Sum2 {
    float hi, lo;
};

// s + t, the rounding errors of the high words kept (Knuth's exact addition).
__device__ __forceinline__ Sum2 add(Sum2 s, Sum2 t) {
    const float hi = __fadd_rn(s.hi, t.hi), b = __fsub_rn(hi, s.hi);
    const float e = __fadd_rn(__fsub_rn(s.hi, __fsub_rn(hi, b)), __fsub_rn(t.hi, b));
    return {hi, __fadd_rn(__fadd_rn(s.lo, t.lo), e)};
}

__device__ __forceinline__ Sum2 square(float x) {
    const float p = __fmul_rn(x, x);
    return {p, __fmaf_rn(x, x, -p)};
}

// The whole CTA's sum, rounded to fp32, on every thread.  part: 32 words that no other call of the row uses.
__device__ __forceinline__ float cta_sum(Sum2 s, Sum2 *part) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        s = add(s, {__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
    const int lane = threadIdx.x & 31, warps = (int)(blockDim.x >> 5);
    if (lane == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = lane < warps ? part[lane] : Sum2{0.0f, 0.0f};
#pragma unroll
    for (int o = 16; o; o >>= 1)
        s = add(s, {__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
    return isinf(s.hi) ? s.hi : __fadd_rn(s.hi, s.lo);
}

__device__ __forceinline__ float inverse_rms(float total, float dim, float eps) {
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(total, dim), eps)));
}

// Eight values as they lie in memory.
template <bool WIDE> struct Raw8 {
    uint4 w[WIDE ? 2 : 1];
};

template <bool WIDE> __device__ __forceinline__ Raw8<WIDE> load_raw(const void *row, uint32_t i) {
    Raw8<WIDE> r;
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(row) + (uint64_t)i * (WIDE ? 4 : 2));
    r.w[0] = p[0];
    if constexpr (WIDE) r.w[1] = p[1];
    return r;
}

template <bool WIDE> __device__ __forceinline__ void values(float (&v)[8], const Raw8<WIDE> &r, bool bf16) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(r.w);
    if constexpr (WIDE) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
    } else if (bf16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(w[e] << 16);
            v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = half_bits_to_float((uint16_t)w[e]);
            v[2 * e + 1] = half_bits_to_float((uint16_t)(w[e] >> 16));
        }
    }
}

// One CTA a row; a thread has chunks of 8 values t, t + T, ..., NS of them.
template <int NS, int MAXT, int MINB, bool HWIDE, bool YWIDE>
__global__ void __launch_bounds__(MAXT, MINB) k_residual_norm(const ResidualNormParams p, int h_type, int y_type) {
    __shared__ Sum2 part[2][32];
    const uint32_t chunks = p.dim / 8, t = threadIdx.x, T = blockDim.x;
    const float dim = (float)p.dim;
    grid_dep_wait();
    for (uint64_t row = blockIdx.x; row < p.n_tok; row += gridDim.x) {
        const uint8_t *yr = static_cast<const uint8_t *>(p.y) + row * p.y_stride * (YWIDE ? 4 : 2);
        const uint8_t *hr = static_cast<const uint8_t *>(p.h) + row * p.h_stride * (HWIDE ? 4 : 2);
        const float *gate = p.gate ? p.gate + row * p.gate_stride : nullptr;
        Raw8<YWIDE> yraw[NS];
        Raw8<HWIDE> hraw[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const uint32_t c = t + s * T;
            if (c < chunks) {
                yraw[s] = load_raw<YWIDE>(yr, c * 8);
                hraw[s] = load_raw<HWIDE>(hr, c * 8);
            }
        }
        float ry = 1.0f;
        if (p.post) {
            Sum2 acc = {0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < NS; ++s)
                if (t + s * T < chunks) {
                    float v[8];
                    values<YWIDE>(v, yraw[s], y_type == Q8_TYPE_BF16);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc = add(acc, square(v[e]));
                }
            ry = inverse_rms(cta_sum(acc, part[0]), dim, p.eps);
        }
        float hv[NS][8];
        Sum2 acc = {0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const uint32_t c = t + s * T;
            if (c >= chunks) continue;
            float u[8], h[8], g[8];
            values<YWIDE>(u, yraw[s], y_type == Q8_TYPE_BF16);
            values<HWIDE>(h, hraw[s], h_type == Q8_TYPE_BF16);
            if (p.post) {
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = __fmul_rn(u[e], ry);
                if (p.gamma_post) {
                    load8(g, p.gamma_post + c * 8);
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[e] = __fmul_rn(u[e], g[e]);
                }
            }
            if (gate) {
                load8s(g, gate + c * 8);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = __fmul_rn(g[e], u[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = __fadd_rn(__fmul_rn(p.residual_scale, h[e]), u[e]);
            if constexpr (!HWIDE) {   // the next norm is of the stored value
                Raw8<false> r;
                uint32_t *w = reinterpret_cast<uint32_t *>(r.w);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = h_type == Q8_TYPE_BF16 ? pack16<true>(h[2 * e], h[2 * e + 1]) : pack16<false>(h[2 * e], h[2 * e + 1]);
                values<false>(h, r, h_type == Q8_TYPE_BF16);
            }
            if (p.h_out) store_out8(p.h_out, h_type, row * p.h_out_stride + c * 8, h, true);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                hv[s][e] = h[e];
                acc = add(acc, square(h[e]));
            }
        }
        if (!p.n_out) {
            if (p.post) __syncthreads();   // part[0] of the next row
            continue;
        }
        const float rh = inverse_rms(cta_sum(acc, part[1]), dim, p.eps);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const uint32_t c = t + s * T;
            if ((c & ~31u) >= chunks) continue;      // whole warps: the quantiser shuffles
            float n[8], g[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) n[e] = c < chunks ? __fmul_rn(hv[s][e], rh) : 0.0f;
            if (p.gamma_next && c < chunks) {
                load8(g, p.gamma_next + c * 8);
#pragma unroll
                for (int e = 0; e < 8; ++e) n[e] = __fmul_rn(n[e], g[e]);
            }
            store_out8(p.n_out, p.n_type, row * p.dim + (uint64_t)c * 8, n, c < chunks);
        }
        __syncthreads();   // part of the next row
    }
}

template <class K>
cudaError_t launch_rows(K kernel, const ResidualNormParams &p, int h_type, int y_type, int threads, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.n_tok < (1u << 30) ? p.n_tok : (1u << 30)));
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
cudaError_t launch_typed(const ResidualNormParams &p, int h_type, int y_type, cudaStream_t st) {
    const uint32_t chunks = p.dim / 8;
    const auto threads = [&](int ns) { return (int)((chunks + ns - 1) / ns + 31) & ~31; };
    if (chunks <= 512) return launch_rows(k_residual_norm<1, 512, 2, HWIDE, YWIDE>, p, h_type, y_type, threads(1), st);
    if (chunks <= 1024) return launch_rows(k_residual_norm<2, 512, 1, HWIDE, YWIDE>, p, h_type, y_type, threads(2), st);
    if (chunks <= 2048) return launch_rows(k_residual_norm<4, 512, 1, HWIDE, YWIDE>, p, h_type, y_type, threads(4), st);
    return launch_rows(k_residual_norm<4, 1024, 1, HWIDE, YWIDE>, p, h_type, y_type, threads(4), st);
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormParams &p, int h_type, int y_type, int, cudaStream_t st) {
    const bool hw = h_type == Q8_TYPE_F32, yw = y_type == Q8_TYPE_F32;
    if (hw) return yw ? launch_typed<true, true>(p, h_type, y_type, st) : launch_typed<true, false>(p, h_type, y_type, st);
    return yw ? launch_typed<false, true>(p, h_type, y_type, st) : launch_typed<false, false>(p, h_type, y_type, st);
}

}  // namespace q8
