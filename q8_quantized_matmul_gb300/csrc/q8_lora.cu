// q8_lora.cu -- low-rank adapters of a few tokens: out[t] = base[t] + s_a B_a (A_a x[t]), a the token's adapter.
//
// k_lora: a cluster of 8 CTAs takes up to T tokens of one adapter and a share of the outputs.  Each CTA multiplies A by its
// eighth of x, the eighths are added through distributed shared memory in a fixed order, and each CTA then has an eighth of
// the share.  One launch and no memory between the two products; fp32 throughout (16-bit weights times fp32, fused
// multiply-adds).  Bound by its chain of trips (ids, rank, A and x, the cluster's barrier, B, store) up to a few MB of
// weights, by the copy rate beyond: B is asked into L2 as soon as the adapter is known.  One token, 4096 to 4096, rank 16: 3.8 us;
// 32 tokens of 32 adapters, 1024 to 32768, Q8_0 x, ranks 1 to 32 of 32: 17 us (30 MB that count, 1.8 TB/s; rows of B are read
// for their rank's part only, but in whole sectors).
#include "q8_lora.cuh"

namespace q8 {
namespace {

constexpr int LC = LORA_CLUSTER; // CTAs of a cluster
constexpr int LT = LORA_THREADS; // threads of a CTA

// Values i .. i + 7 (i a multiple of 8) of a token's x.
__device__ __forceinline__ void x8(float (&v)[8], const LoraParams &p, uint64_t tok, uint32_t i) {
    if (p.x_type == Q8_TYPE_F32) {
        load8s(v, static_cast<const float *>(p.x) + tok * p.x_stride + i);
    } else if (p.x_type == Q8_TYPE_Q8_0) {
        const uint16_t *blk = reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(p.x) +
                                                                 (tok * (p.in_dim / QK) + i / QK) * QB);
        const float d = half_bits_to_float(blk[0]);
        const uint16_t *q = blk + 1 + (i % QK) / 2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[4];
            quants4(f, q[2 * h] | (uint32_t)q[2 * h + 1] << 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * h + e] = f[e] * d;
        }
    } else {
        values16(v, *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + tok * p.x_stride + i),
                 p.x_type == Q8_TYPE_BF16);
    }
}

// Sums of N values over the warp; lane l ends with the sum of value l / (32 / N), N a power of two up to 32.
template <int N> __device__ __forceinline__ float warp_sums(float (&v)[N]) {
    const uint32_t lane = threadIdx.x & 31u;
    int b = 16;
#pragma unroll
    for (int w = N / 2; w; w >>= 1, b >>= 1) {
        const bool up = lane & (uint32_t)b;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float give = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, b);
        }
    }
    float s = v[0];
#pragma unroll
    for (; b; b >>= 1) s += __shfl_xor_sync(0xffffffffu, s, b);
    return s;
}

struct Shared {
    float part[LORA_GROUP][LORA_MAX_RANK];
    float low[LORA_GROUP][LORA_MAX_RANK];   // read 16 bytes at a time
    uint32_t tok[LORA_GROUP];
    uint32_t n, pos;
};

// Share `share` of `shares` of the outputs of n tokens of adapter id, by the whole cluster (this CTA is its k-th).
// T: most tokens; RR: rows of A that a warp takes at a time; U: outputs that a thread takes at a time.
template <int T, int RR, int U>
__device__ __forceinline__ void group_share(const LoraParams &p, Shared &sh, int32_t id, uint32_t rank, uint32_t n, const uint32_t (&mine)[T],
                                            uint32_t share, uint32_t shares, uint32_t k) {
    const uint32_t t = threadIdx.x, lane = t & 31u, warp = t >> 5;
    const uint32_t o0 = (uint32_t)((uint64_t)p.out_dim * (share * LC + k) / (shares * LC)),
                   o1 = (uint32_t)((uint64_t)p.out_dim * (share * LC + k + 1) / (shares * LC));
    const float scale = p.scales ? p.scales[id] : 1.0f;
    const uint16_t *b = p.b + (uint64_t)id * p.b_stride;
    if (t == 0 && o1 > o0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(b + (uint64_t)o0 * p.max_rank), "r"((o1 - o0) * p.max_rank * 2) : "memory");
    // ---- A times this CTA's eighth of x
    const uint16_t *a = p.a + (uint64_t)id * p.a_stride;
    const uint32_t nb = p.in_dim / QK, i0 = (uint32_t)((uint64_t)nb * k / LC) * QK, i1 = (uint32_t)((uint64_t)nb * (k + 1) / LC) * QK;
    for (uint32_t r0 = warp; r0 < rank; r0 += RR * (LT / 32)) {
        float acc[T * RR];
#pragma unroll
        for (int i = 0; i < T * RR; ++i) acc[i] = 0.0f;
#pragma unroll 2
        for (uint32_t i = i0 + lane * 8; i < i1; i += 256) {
            uint4 raw[RR];
#pragma unroll
            for (int q = 0; q < RR; ++q) {
                raw[q] = make_uint4(0, 0, 0, 0);
                if (r0 + q * (LT / 32) < rank) raw[q] = __ldg(reinterpret_cast<const uint4 *>(a + (uint64_t)(r0 + q * (LT / 32)) * p.in_dim + i));
            }
#pragma unroll
            for (int m = 0; m < T; ++m) {
                if (m >= n) continue;
                float x[8];
                x8(x, p, mine[m], i);
#pragma unroll
                for (int q = 0; q < RR; ++q) {
                    float w[8];
                    values16(w, raw[q], p.bf16);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[m * RR + q] = fmaf(w[e], x[e], acc[m * RR + q]);
                }
            }
        }
        const float s = warp_sums<T * RR>(acc);
        const uint32_t v = lane / (32 / (T * RR)), r = r0 + v % RR * (LT / 32);
        if (lane % (32 / (T * RR)) == 0 && r < rank) sh.part[v / RR][r] = s;
    }
    cluster_arrive();
    cluster_wait();
    const uint32_t ranks8 = (rank + 7) & ~7u;
    for (uint32_t i = t; i < n * ranks8; i += LT) {
        const uint32_t m = i / ranks8, r = i - m * ranks8;
        float v = 0.0f;
        if (r < rank) {
            float f[LC];
#pragma unroll
            for (uint32_t q = 0; q < LC; ++q) f[q] = ld_cluster(cluster_addr(&sh.part[m][r], q));
#pragma unroll
            for (uint32_t q = 0; q < LC; ++q) v += f[q];
            v *= scale;
        }
        sh.low[m][r] = v;
    }
    cluster_arrive();   // the other CTAs may go on once all have read
    __syncthreads();
    // ---- this CTA's outputs
    for (uint32_t ob = o0 + t; ob < o1; ob += U * LT) {
        float acc[U][T], base[U][T];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int m = 0; m < T; ++m) {
                acc[u][m] = base[u][m] = 0.0f;
                if (p.base && m < n && ob + u * LT < o1) base[u][m] = p.base[(uint64_t)mine[m] * p.base_stride + ob + u * LT];
            }
#pragma unroll 2
        for (uint32_t c = 0; c < ranks8 / 8; ++c) {
            uint4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                raw[u] = make_uint4(0, 0, 0, 0);
                if (ob + u * LT < o1) raw[u] = __ldg(reinterpret_cast<const uint4 *>(b + (uint64_t)(ob + u * LT) * p.max_rank) + c);
            }
            if (c * 8 + 8 > rank) {
#pragma unroll
                for (int u = 0; u < U; ++u) raw[u] = first_values(raw[u], (int)rank - (int)c * 8);
            }
#pragma unroll
            for (int m = 0; m < T; ++m) {
                if (m >= n) continue;
                float h[8];
                load8s(h, &sh.low[m][c * 8]);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float w[8];
                    values16(w, raw[u], p.bf16);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[u][m] = fmaf(w[e], h[e], acc[u][m]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int m = 0; m < T; ++m)
                if (m < n && ob + u * LT < o1) p.out[(uint64_t)mine[m] * p.out_stride + ob + u * LT] = base[u][m] + acc[u][m];
    }
    cluster_wait();
}

// A lone token takes more rows and outputs at a time.
template <int T>
__device__ __forceinline__ void share_of(const LoraParams &p, Shared &sh, int32_t id, uint32_t rank, uint32_t n, const uint32_t (&mine)[T],
                                         uint32_t share, uint32_t shares, uint32_t k) {
    const uint32_t first[1] = {mine[0]};
    if (T == 1) group_share<1, 4, 2>(p, sh, id, rank, 1, first, share, shares, k);
    else if (n == 1) group_share<1, 4, 4>(p, sh, id, rank, 1, first, share, shares, k);
    else group_share<T, 2, 2>(p, sh, id, rank, n, mine, share, shares, k);
}

// A cluster (p.splits of them) a token: those of a group's tokens share its outputs.
template <int T> __global__ void __cluster_dims__(LC, 1, 1) __launch_bounds__(LT, 4) k_lora(const LoraParams p) {
    __shared__ __align__(16) Shared sh;
    const uint32_t t = threadIdx.x, lane = t & 31u, warp = t >> 5, k = cluster_rank();
    const uint32_t cluster = blockIdx.x / LC, j = cluster / p.splits, split = cluster - j * p.splits;
    grid_dep_wait();
    const int32_t id = p.adapter_of[j];
    if (id < 0 || (uint32_t)id >= p.n_adapters) {
        if (id >= 0 && t == 0) raise_error(p.err, DEV_ERANGE);
        if (p.base != p.out) {
            const uint32_t share = split * LC + k, shares = p.splits * LC;
            const uint32_t o1 = (uint32_t)((uint64_t)p.out_dim * (share + 1) / shares);
#pragma unroll 4
            for (uint32_t o = (uint32_t)((uint64_t)p.out_dim * share / shares) + t; o < o1; o += LT)
                p.out[j * p.out_stride + o] = p.base ? __ldg(p.base + j * p.base_stride + o) : 0.0f;
        }
        return;
    }
    const uint32_t rank = cut_rank(p, given_rank(p, id), t == 0);
    uint32_t n = 1, pos = 0, mine[T] = {j};
    if (T > 1) {
        // groups are T tokens of the adapter in their order: j's place in its group, and the others
        if (warp == 0) {
            uint32_t before = 0;
            for (uint32_t i = 0; i < j; i += 32)
                before += __popc(__ballot_sync(0xffffffffu, i + lane < j && p.adapter_of[i + lane] == id));
            const uint32_t first = before - before % T;      // of the adapter's tokens, the group's first
            uint32_t m = 0;
            for (uint32_t i = 0; i < p.n_tok && m < first + T; i += 32) {
                const bool hit = i + lane < p.n_tok && p.adapter_of[i + lane] == id;
                const uint32_t mask = __ballot_sync(0xffffffffu, hit), at = m + __popc(mask & ((1u << lane) - 1u));
                if (hit && at >= first && at < first + T) sh.tok[at - first] = i + lane;
                m += __popc(mask);
            }
            if (lane == 0) {
                sh.n = min(m - first, (uint32_t)T);
                sh.pos = before - first;
            }
        }
        __syncthreads();
        n = sh.n;
        pos = sh.pos;
#pragma unroll
        for (int m = 0; m < T; ++m) mine[m] = m < n ? sh.tok[m] : 0;
    }
    share_of<T>(p, sh, id, rank, n, mine, split * n + pos, p.splits * n, k);
}

// The groups of the list that k_lora_route made: adapters with too few tokens for a tile.
__global__ void __cluster_dims__(LC, 1, 1) __launch_bounds__(LT, 4) k_lora_groups(const LoraParams p) {
    __shared__ __align__(16) Shared sh;
    const uint32_t k = cluster_rank(), cluster = blockIdx.x / LC, clusters = gridDim.x / LC;
    grid_dep_wait();
    const uint32_t n_groups = (uint32_t)p.tiles[0].y;
    if (n_groups == 0) return;
    // several clusters a group where there are more clusters than groups, of at least a thread an output
    const uint32_t most = (p.out_dim + LT * LC - 1) / (LT * LC), shares = max(1u, min(most, clusters / n_groups));
    for (uint32_t i = cluster; i < n_groups * shares; i += clusters) {
        const int4 g = p.groups[i / shares];                 // {adapter, first of perm, tokens, rank}
        uint32_t mine[LORA_GROUP];
#pragma unroll
        for (int m = 0; m < (int)LORA_GROUP; ++m) mine[m] = m < g.z ? p.perm[g.y + m] : 0;
        share_of<LORA_GROUP>(p, sh, g.x, (uint32_t)g.w, (uint32_t)g.z, mine, i % shares, shares, k);
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_lora(const LoraParams &q, int num_sms, cudaStream_t st) {
    LoraParams p = q;
    p.splits = lora_splits(p.n_tok, p.out_dim, num_sms);
    const dim3 grid((unsigned)((uint64_t)LC * p.splits * p.n_tok));
    if (p.n_tok == 1) return launch_dependent(k_lora<1>, p, grid, LT, 0, st);
    return launch_dependent(k_lora<LORA_GROUP>, p, grid, LT, 0, st);
}

cudaError_t launch_lora_groups(const LoraParams &p, int num_sms, cudaStream_t st) {
    const unsigned fit = (unsigned)num_sms * 4 / LC;
    return launch_dependent(k_lora_groups, p, dim3(fit * LC), LT, 0, st);
}

}  // namespace q8
