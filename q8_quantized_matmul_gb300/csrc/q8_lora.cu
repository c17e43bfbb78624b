// q8_lora.cu -- low-rank adapters of many requests: out[t] = base[t] + s_a B_a (A_a x[t]), a the token's adapter.
//
// k_lora: a cluster of 8 CTAs takes up to T tokens of one adapter.  Each CTA multiplies A by its eighth of x, the
// eighths are added through distributed shared memory in a fixed order, and each CTA then has its share of the outputs.
// One launch and no memory between the two products; fp32 throughout (16-bit weights times fp32, fused multiply-adds).
#include "q8_lora.cuh"

namespace q8 {
namespace {

constexpr int LC = 8;            // CTAs of a cluster
constexpr int LT = 256;          // threads of a CTA
constexpr uint32_t XS = 1024;    // values of x that a CTA holds at a time

// Values i .. i + 7 (i a multiple of 8) of a token's x.
__device__ __forceinline__ void x8(float (&v)[8], const LoraParams &p, uint64_t tok, uint32_t i) {
    if (p.x_type == Q8_TYPE_F32) {
        load8s(v, static_cast<const float *>(p.x) + tok * p.x_stride + i);
    } else if (p.x_type == Q8_TYPE_Q8_0) {
        const uint16_t *blk = reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(p.x) +
                                                                 (tok * (p.in_dim / QK) + i / QK) * QB);
        const float d = half_bits_to_float(blk[0]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t q = blk[1 + (i % QK) / 2 + e];
            v[2 * e] = (float)(int8_t)q * d;
            v[2 * e + 1] = (float)(int8_t)(q >> 8) * d;
        }
    } else {
        values16(v, *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + tok * p.x_stride + i),
                 p.x_type == Q8_TYPE_BF16);
    }
}

template <int T> __global__ void __cluster_dims__(LC, 1, 1) __launch_bounds__(LT) k_lora(const LoraParams p) {
    __shared__ __align__(16) float xs[2][T][XS / 2];   // values 0..3 and 4..7 of each 8 apart: no bank conflicts
    __shared__ float part[T][LORA_MAX_RANK];
    __shared__ __align__(16) float low[T][LORA_MAX_RANK];
    __shared__ uint32_t tok[T];
    __shared__ uint32_t n_mine;
    const uint32_t t = threadIdx.x, lane = t & 31u, warp = t >> 5, k = cluster_rank();
    const uint32_t cluster = blockIdx.x / LC, j = cluster / p.splits, split = cluster - j * p.splits;
    grid_dep_wait();
    const int32_t id = p.adapter_of[j];
    const uint32_t share = split * LC + k, shares = p.splits * LC;
    const uint32_t o0 = (uint32_t)((uint64_t)p.out_dim * share / shares), o1 = (uint32_t)((uint64_t)p.out_dim * (share + 1) / shares);
    if (id < 0 || (uint32_t)id >= p.n_adapters) {
        if (id >= 0 && t == 0) raise_error(p.err, DEV_ERANGE);
        if (p.base != p.out)
            for (uint32_t o = o0 + t; o < o1; o += LT)
                p.out[j * p.out_stride + o] = p.base ? p.base[j * p.base_stride + o] : 0.0f;
        return;
    }
    // the tokens of this adapter before j: every T-th starts a group
    uint32_t before = 0;
    for (uint32_t i = 0; i < j; i += LT) before += (uint32_t)__syncthreads_count(i + t < j && p.adapter_of[i + t] == id);
    if (before % T) return;
    if (warp == 0) {
        uint32_t m = 0;
        for (uint32_t i = j; i < p.n_tok && m < T; i += 32) {
            const bool hit = i + lane < p.n_tok && p.adapter_of[i + lane] == id;
            const uint32_t mask = __ballot_sync(0xffffffffu, hit), at = m + __popc(mask & ((1u << lane) - 1u));
            if (hit && at < T) tok[at] = i + lane;
            m += __popc(mask);
        }
        if (lane == 0) n_mine = min(m, (uint32_t)T);
    }
    const uint32_t rank = rank_of(p, id, t == 0);
    for (uint32_t i = t; i < T * LORA_MAX_RANK; i += LT) part[i / LORA_MAX_RANK][i % LORA_MAX_RANK] = 0.0f;
    __syncthreads();
    const uint32_t n = n_mine;
    const uint16_t *a = p.a + (uint64_t)id * p.a_stride;
    const uint32_t nb = p.in_dim / QK, i0 = (uint32_t)((uint64_t)nb * k / LC) * QK, i1 = (uint32_t)((uint64_t)nb * (k + 1) / LC) * QK;
    for (uint32_t s0 = i0; s0 < i1; s0 += XS) {
        const uint32_t len = min(XS, i1 - s0), chunks = len / 8;
        for (uint32_t i = t; i < n * chunks; i += LT) {
            const uint32_t m = i / chunks, c = i - m * chunks;
            float v[8];
            x8(v, p, tok[m], s0 + c * 8);
            *reinterpret_cast<float4 *>(&xs[0][m][c * 4]) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(&xs[1][m][c * 4]) = make_float4(v[4], v[5], v[6], v[7]);
        }
        __syncthreads();
        for (uint32_t r = warp; r < rank; r += LT / 32) {
            const uint16_t *row = a + (uint64_t)r * p.in_dim + s0;
            float acc[T];
#pragma unroll
            for (int m = 0; m < T; ++m) acc[m] = 0.0f;
#pragma unroll 2
            for (uint32_t c = lane; c < chunks; c += 32) {
                float w[8];
                values16(w, __ldg(reinterpret_cast<const uint4 *>(row + c * 8)), p.bf16);
#pragma unroll
                for (int m = 0; m < T; ++m)
                    if (m < n) {
                        const float4 u = *reinterpret_cast<const float4 *>(&xs[0][m][c * 4]);
                        const float4 v = *reinterpret_cast<const float4 *>(&xs[1][m][c * 4]);
                        acc[m] = fmaf(w[0], u.x, acc[m]);
                        acc[m] = fmaf(w[1], u.y, acc[m]);
                        acc[m] = fmaf(w[2], u.z, acc[m]);
                        acc[m] = fmaf(w[3], u.w, acc[m]);
                        acc[m] = fmaf(w[4], v.x, acc[m]);
                        acc[m] = fmaf(w[5], v.y, acc[m]);
                        acc[m] = fmaf(w[6], v.z, acc[m]);
                        acc[m] = fmaf(w[7], v.w, acc[m]);
                    }
            }
#pragma unroll
            for (int m = 0; m < T; ++m) {
#pragma unroll
                for (int o = 16; o; o >>= 1) acc[m] += __shfl_xor_sync(0xffffffffu, acc[m], o);
                if (lane == 0 && m < n) part[m][r] += acc[m];
            }
        }
        __syncthreads();
    }
    cluster_arrive();
    cluster_wait();
    const float scale = p.scales ? p.scales[id] : 1.0f;
    const uint32_t ranks8 = (rank + 7) & ~7u;
    for (uint32_t i = t; i < n * ranks8; i += LT) {
        const uint32_t m = i / ranks8, r = i - m * ranks8;
        float v = 0.0f;
        if (r < rank) {
#pragma unroll
            for (uint32_t q = 0; q < LC; ++q) v += ld_cluster(cluster_addr(&part[m][r], q));
            v *= scale;
        }
        low[m][r] = v;
    }
    cluster_arrive();   // the other CTAs may leave once all have read
    __syncthreads();
    const uint16_t *b = p.b + (uint64_t)id * p.b_stride;
    for (uint32_t o = o0 + t; o < o1; o += LT) {
        float acc[T];
#pragma unroll
        for (int m = 0; m < T; ++m) acc[m] = 0.0f;
        const uint4 *row = reinterpret_cast<const uint4 *>(b + (uint64_t)o * p.max_rank);
        for (uint32_t c = 0; c < ranks8 / 8; ++c) {
            float w[8];
            values16(w, __ldg(row + c), p.bf16);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = c * 8 + e < rank ? w[e] : 0.0f;
#pragma unroll
            for (int m = 0; m < T; ++m)
                if (m < n) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[m] = fmaf(w[e], low[m][c * 8 + e], acc[m]);
                }
        }
#pragma unroll
        for (int m = 0; m < T; ++m)
            if (m < n) {
                const uint64_t row_of = tok[m];
                p.out[row_of * p.out_stride + o] = (p.base ? p.base[row_of * p.base_stride + o] : 0.0f) + acc[m];
            }
    }
    cluster_wait();
}

}  // namespace

cudaError_t launch_lora(const LoraParams &q, int num_sms, cudaStream_t st) {
    LoraParams p = q;
    const uint32_t most = (p.out_dim + LT * LC - 1) / (LT * LC), want = (uint32_t)(2 * num_sms) / (p.n_tok * LC);
    p.splits = want < 1 ? 1 : want > most ? most : want;
    return launch_dependent(k_lora<4>, p, dim3((unsigned)((uint64_t)LC * p.splits * p.n_tok)), LT, 0, st);
}

}  // namespace q8
