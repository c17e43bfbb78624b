// q8_lora_tc.cu -- low-rank adapters of many tokens on the tensor cores: out[t] = base[t] + s_a B_a (A_a x[t]).
//
//   k_lora_route   one CTA orders the tokens by adapter and cuts them into tiles of up to 128 tokens of one adapter.  The
//                  order inside an adapter is left to chance: a token's result does not depend on its place in a tile.
//   k_lora_shrink  a cluster of 8 CTAs a tile, each an eighth of in_dim: low = A x with the tokens along the rows of the
//                  product.  The eighths are added through distributed shared memory in a fixed order.
//   k_lora_expand  tiles of 128 outputs (rows) by the tile's tokens (columns): a warp's lanes hold neighbouring outputs of one
//                  token, so base and out are read and written in whole lines.
//
// fp32 accuracy from 16-bit products: an fp32 value is the exact sum of three bf16 terms (24 bits; each rounds what the ones
// before left), an fp16 weight of two, and a product of two bf16 is exact in the fp32 accumulators.  Terms below 2^-24 of the
// product are left out.  The first terms' products and the rest are summed apart, for the tensor cores drop what is shifted
// out of a sum.  bf16 x takes one term, fp16 x two (one and kind f16 with fp16 adapters).
#include "q8_launch.h"
#include "q8_lora.cuh"
#include "q8_tcgen05.cuh"

namespace q8 {
namespace {

constexpr uint32_t TM = 128;              // tokens of a tile
constexpr uint32_t KB = 64;               // values of a K step: a 128-byte row of 16-bit terms
constexpr uint32_t PLANE = TM * 128;      // bytes of one term's 128 x 64 tile
constexpr int SC = 8;                     // CTAs of a cluster of k_lora_shrink
constexpr int TT = 256;
constexpr int NO_ADAPTER = -1;

// ---------------------------------------------------------------- route
constexpr int RT = 1024;

// Inclusive sums of two values over the CTA; totals on every thread.
__device__ __forceinline__ void scan2(int &a, int &b, int &ta, int &tb, int2 *warps) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) a += x, b += y;
    }
    if (lane == 31) warps[w] = make_int2(a, b);
    __syncthreads();
    if (w == 0) {
        int2 v = warps[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
            if (lane >= o) v.x += x, v.y += y;
        }
        warps[lane] = v;
    }
    __syncthreads();
    if (w) a += warps[w - 1].x, b += warps[w - 1].y;
    ta = warps[31].x;
    tb = warps[31].y;
}

// Bucket of token i: its adapter, n_adapters for none (-1: nothing to do for it either, base is out).
__device__ __forceinline__ int bucket_of(const LoraParams &p, uint32_t i, bool tell) {
    const int32_t id = p.adapter_of[i];
    if (id >= 0 && (uint32_t)id < p.n_adapters && rank_of(p, id, tell) > 0) return id;
    if (tell && id >= 0 && (uint32_t)id >= p.n_adapters) raise_error(p.err, DEV_ERANGE);
    return p.base == p.out ? -1 : (int)p.n_adapters;
}

__global__ void __launch_bounds__(RT) k_lora_route(const LoraParams p) {
    extern __shared__ int counts[];       // [n_adapters + 1]: tokens, then the next free place
    __shared__ int2 warps[32];
    const int n = (int)p.n_adapters + 1, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < n; i += RT) counts[i] = 0;
    grid_dep_wait();
    __syncthreads();
    const uint32_t rounds = (p.n_tok + RT - 1) / RT;
    for (uint32_t r = 0; r < rounds; ++r) {
        const uint32_t i = r * RT + threadIdx.x;
        const int b = i < p.n_tok ? bucket_of(p, i, true) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, b);
        if (b >= 0 && lane == __ffs(same) - 1) atomicAdd(&counts[b], __popc(same));
    }
    __syncthreads();
    const int per = (n + RT - 1) / RT, b0 = min(n, (int)threadIdx.x * per), b1 = min(n, b0 + per);
    int tokens = 0, tiles = 0, all, n_tiles;
    for (int b = b0; b < b1; ++b) {
        tokens += counts[b];
        tiles += (counts[b] + (int)TM - 1) / (int)TM;
    }
    int t = tokens, k = tiles;
    scan2(t, k, all, n_tiles, warps);
    t -= tokens;
    k -= tiles;
    for (int b = b0; b < b1; ++b) {
        const int c = counts[b];
        counts[b] = t;
        const bool bare = b == (int)p.n_adapters;
        const int rank = bare || c == 0 ? 0 : (int)rank_of(p, b, false);
        for (int at = 0; at < c; at += TM, ++k)
            p.tiles[1 + k] = make_int4(bare ? NO_ADAPTER : b, t + at, min((int)TM, c - at), rank);
        t += c;
    }
    if (threadIdx.x == 0) p.tiles[0] = make_int4(n_tiles, 0, 0, 0);
    __syncthreads();
    for (uint32_t r = 0; r < rounds; ++r) {
        const uint32_t i = r * RT + threadIdx.x;
        const int b = i < p.n_tok ? bucket_of(p, i, false) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, b);
        int at = 0;
        if (b >= 0 && lane == __ffs(same) - 1) at = atomicAdd(&counts[b], __popc(same));
        at = __shfl_sync(0xffffffffu, at, __ffs(same) - 1) + __popc(same & ((1u << lane) - 1u));
        if (b >= 0) p.perm[at] = i;
    }
}

// ---------------------------------------------------------------- terms
// Two fp32 values as N packed bf16 pairs that sum to them (each rounds what is left).
template <int N> __device__ __forceinline__ void terms2(uint32_t (&t)[N], float a, float b) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        t[i] = pack16<true>(a, b);
        if (i + 1 < N) {
            a = __fsub_rn(a, __uint_as_float(t[i] << 16));
            b = __fsub_rn(b, __uint_as_float(t[i] & 0xffff0000u));
        }
    }
}

// Eight fp16 values as N chunks of bf16 terms.
template <int N> __device__ __forceinline__ void terms_f16(uint4 (&out)[N], const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t t[N];
        terms2<N>(t, half_bits_to_float((uint16_t)w[e]), half_bits_to_float((uint16_t)(w[e] >> 16)));
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<uint32_t *>(&out[i])[e] = t[i];
    }
}

// Byte offset of 16-byte chunk c of row r in a tile of 128-byte rows, swizzled as the matrix descriptors say.
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t c) { return r * 128 + ((c ^ (r & 7u)) << 4); }

// The products of one K step: x terms times weight terms, those that reach 2^-24.  x, w: the terms' tiles, x_step and w_step
// bytes apart.  Term (0, 0) goes to d; the others to d + rest, or with rest 0 to d as well.  acc, acc_rest: whether the
// accumulators hold sums already.
template <int NX, int NW, bool X_IS_A>
__device__ __forceinline__ void issue_terms(uint32_t d, uint32_t rest, uint32_t x, uint32_t x_step, uint32_t w, uint32_t w_step,
                                            int ksteps, uint32_t idesc, bool acc, bool acc_rest) {
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            if (i + j > 2) continue;
            const uint64_t xd = sw128_desc(x + i * x_step), wd = sw128_desc(w + j * w_step);
            const bool apart = i + j && rest;
            for (int k = 0; k < ksteps; ++k) {
                tc_mma_f16(apart ? d + rest : d, (X_IS_A ? xd : wd) + 2 * k, (X_IS_A ? wd : xd) + 2 * k, idesc, apart ? acc_rest : acc);
                if (apart) acc_rest = true;
                else acc = true;
            }
        }
}

__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}

// ---------------------------------------------------------------- shrink
enum XKind { X_F32, X_Q8, X_RAW, X_F16 };   // RAW: 16-bit values as they are; F16: split into two bf16 terms

// What a thread holds of a K step of x: four values of each of 8 rows, or eight values of each of 4.
template <int XK> struct XRegs {
    static constexpr int ROWS = XK == X_F32 || XK == X_Q8 ? 8 : 4;
    uint4 v[ROWS];
};
template <> struct XRegs<X_Q8> {
    static constexpr int ROWS = 8;
    uint32_t q[8];
    uint16_t d[8];
};

template <int XK>
__device__ __forceinline__ void load_x(XRegs<XK> &r, const LoraParams &p, const uint32_t (&tok)[XRegs<XK>::ROWS], uint32_t k0) {
    constexpr bool FOUR = XRegs<XK>::ROWS == 8;
    const uint32_t k = k0 + (FOUR ? threadIdx.x % 16 * 4 : threadIdx.x % 8 * 8);
    const bool in = k < p.in_dim;
#pragma unroll
    for (int i = 0; i < XRegs<XK>::ROWS; ++i) {
        const bool live = in && tok[i] != 0xffffffffu;
        if constexpr (XK == X_Q8) {
            r.q[i] = 0;
            r.d[i] = 0;
            if (live) {
                const uint16_t *b = reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(p.x) +
                                                                       ((uint64_t)tok[i] * (p.in_dim / QK) + k / QK) * QB);
                r.d[i] = __ldg(b);
                r.q[i] = __ldg(b + 1 + k % QK / 2) | (uint32_t)__ldg(b + 2 + k % QK / 2) << 16;
            }
        } else {
            r.v[i] = make_uint4(0, 0, 0, 0);
            if (live)
                r.v[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.x) +
                                                               ((uint64_t)tok[i] * p.x_stride + k) * (XK == X_F32 ? 4 : 2)));
        }
    }
}

template <int XK, int NX> __device__ __forceinline__ void store_x(uint8_t *tile, const XRegs<XK> &r) {
    constexpr bool FOUR = XRegs<XK>::ROWS == 8;
    const uint32_t t = threadIdx.x;
#pragma unroll
    for (int i = 0; i < XRegs<XK>::ROWS; ++i) {
        if constexpr (FOUR) {
            const uint32_t row = t / 16 + 16 * i, at = swizzled(row, t % 16 / 2) + t % 2 * 8;
            float v[4];
            if constexpr (XK == X_F32) {
                v[0] = __uint_as_float(r.v[i].x);
                v[1] = __uint_as_float(r.v[i].y);
                v[2] = __uint_as_float(r.v[i].z);
                v[3] = __uint_as_float(r.v[i].w);
            } else {
                const float d = half_bits_to_float(r.d[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = (float)(int8_t)(r.q[i] >> (8 * e)) * d;
            }
            uint32_t a[NX], b[NX];
            terms2<NX>(a, v[0], v[1]);
            terms2<NX>(b, v[2], v[3]);
#pragma unroll
            for (int j = 0; j < NX; ++j) *reinterpret_cast<uint2 *>(tile + j * PLANE + at) = make_uint2(a[j], b[j]);
        } else {
            const uint32_t row = t / 8 + 32 * i, at = swizzled(row, t % 8);
            uint4 c[NX];
            if constexpr (XK == X_F16) terms_f16<NX>(c, r.v[i]);
            else c[0] = r.v[i];
#pragma unroll
            for (int j = 0; j < NX; ++j) *reinterpret_cast<uint4 *>(tile + j * PLANE + at) = c[j];
        }
    }
}

// The weights' rows of a K step, 8 values of rows t / 8, t / 8 + 32, ...
struct WRegs {
    uint4 v[LORA_MAX_RANK / 32];
};
__device__ __forceinline__ void load_w(WRegs &r, const LoraParams &p, const uint16_t *a, uint32_t rank, uint32_t k0) {
    const uint32_t k = k0 + threadIdx.x % 8 * 8;
#pragma unroll
    for (uint32_t i = 0; i < LORA_MAX_RANK / 32; ++i) {
        const uint32_t row = threadIdx.x / 8 + 32 * i;
        r.v[i] = make_uint4(0, 0, 0, 0);
        if (row < rank && k < p.in_dim) r.v[i] = __ldg(reinterpret_cast<const uint4 *>(a + (uint64_t)row * p.in_dim + k));
    }
}
template <int NW> __device__ __forceinline__ void store_w(uint8_t *tile, uint32_t step, const WRegs &r, uint32_t rows) {
#pragma unroll
    for (uint32_t i = 0; i < LORA_MAX_RANK / 32; ++i) {
        const uint32_t row = threadIdx.x / 8 + 32 * i;
        if (row >= rows) continue;
        uint4 c[NW];
        if constexpr (NW == 2) terms_f16<NW>(c, r.v[i]);
        else c[0] = r.v[i];
#pragma unroll
        for (int j = 0; j < NW; ++j) *reinterpret_cast<uint4 *>(tile + j * step + swizzled(row, threadIdx.x % 8)) = c[j];
    }
}

__host__ __device__ constexpr uint32_t round16(uint32_t r) { return (r + 15u) & ~15u; }

template <int NX, int NW> __host__ __device__ constexpr uint32_t shrink_stage(uint32_t max_rank) {
    return NX * PLANE + NW * round16(max_rank) * 128;
}
template <int NX, int NW> __host__ __device__ constexpr uint32_t shrink_smem(uint32_t max_rank) {
    const uint32_t two = 2 * shrink_stage<NX, NW>(max_rank), part = TM * (round16(max_rank) + 4) * 4;
    return 1024 + (two > part ? two : part);
}

template <int XK, int NX, int NW>
__global__ void __cluster_dims__(SC, 1, 1) __launch_bounds__(TT) k_lora_shrink(const LoraParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    __shared__ uint64_t done[2];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t t = threadIdx.x, warp = t >> 5, k = cluster_rank();
    const uint32_t cols_max = round16(p.max_rank), w_step = cols_max * 128, stage = shrink_stage<NX, NW>(p.max_rank);
    const uint32_t tmem_cols = cols_max <= 16 ? 32 : cols_max <= 32 ? 64 : cols_max <= 64 ? 128 : 256, rest = tmem_cols / 2;
    if (t == 0) {
        mbar_init(&done[0], 1);
        mbar_init(&done[1], 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    grid_dep_wait();
    if (warp == 0) tmem_alloc(&tmem_slot, tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int n_tiles = p.tiles[0].x;
    const uint32_t nb = (p.in_dim + KB - 1) / KB, kb0 = nb * k / SC, kb1 = nb * (k + 1) / SC;
    uint32_t u = 0;                                          // K steps so far
    for (int tile = blockIdx.x / SC; tile < n_tiles; tile += gridDim.x / SC) {
        const int4 T = p.tiles[1 + tile];
        if (T.x == NO_ADAPTER) continue;
        const uint32_t count = T.z, rank = T.w, cols = round16(rank);
        const uint16_t *a = p.a + (uint64_t)T.x * p.a_stride;
        const uint32_t idesc = tc_idesc(TM, cols, !(XK == X_RAW && !p.bf16 && NW == 1));
        uint32_t tok[XRegs<XK>::ROWS];
#pragma unroll
        for (int i = 0; i < XRegs<XK>::ROWS; ++i) {
            const uint32_t row = XRegs<XK>::ROWS == 8 ? t / 16 + 16 * i : t / 8 + 32 * i;
            tok[i] = row < count ? p.perm[T.y + row] : 0xffffffffu;
        }
        XRegs<XK> x;
        WRegs w;
        if (kb0 < kb1) {
            load_x<XK>(x, p, tok, kb0 * KB);
            load_w(w, p, a, rank, kb0 * KB);
        }
        for (uint32_t b = kb0; b < kb1; ++b, ++u) {
            XRegs<XK> xn;
            WRegs wn;
            if (b + 1 < kb1) {
                load_x<XK>(xn, p, tok, (b + 1) * KB);
                load_w(wn, p, a, rank, (b + 1) * KB);
            }
            uint8_t *s = smem + (u & 1) * stage;
            if (u >= 2) tile_wait(&done[u & 1], (u / 2 - 1) & 1, p.err, &abort_flag);
            store_x<XK, NX>(s, x);
            store_w<NW>(s + NX * PLANE, w_step, w, cols);
            fence_async_smem();
            __syncthreads();
            if (warp == 0 && elect_one()) {
                tc_fence_after();
                issue_terms<NX, NW, true>(tmem, rest, smem_addr(s), PLANE, smem_addr(s) + NX * PLANE, w_step, KB / 16, idesc, b != kb0, b != kb0);
                tc_commit(&done[u & 1]);
            }
            if (b + 1 < kb1) {
                x = xn;
                w = wn;
            }
        }
        // this CTA's sums, one row a thread
        float *part = reinterpret_cast<float *>(smem);
        const uint32_t pitch = cols + 4;
        if (kb0 < kb1) {
            tile_wait(&done[(u - 1) & 1], ((u - 1) / 2) & 1, p.err, &abort_flag);
            tc_fence_after();
        }
        __syncthreads();
        const uint32_t row = (warp & 3) * 32 + (t & 31);
        for (uint32_t c = (warp >> 2) * 16; c < cols; c += 32) {
            uint32_t d0[16], d1[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) d0[e] = d1[e] = 0;
            if (kb0 < kb1) {
                const uint32_t at = tmem + ((warp & 3) << 21) + c;
                tc_ld16(at, d0);
                if constexpr (NX + NW > 2) tc_ld16(at + rest, d1);
                tc_wait_ld();
                tc_regs_ready(d0);
                tc_regs_ready(d1);
            }
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                float4 v = make_float4(__uint_as_float(d0[e]), __uint_as_float(d0[e + 1]), __uint_as_float(d0[e + 2]), __uint_as_float(d0[e + 3]));
                if constexpr (NX + NW > 2) {
                    v.x += __uint_as_float(d1[e]);
                    v.y += __uint_as_float(d1[e + 1]);
                    v.z += __uint_as_float(d1[e + 2]);
                    v.w += __uint_as_float(d1[e + 3]);
                }
                *reinterpret_cast<float4 *>(part + row * pitch + c + e) = v;
            }
        }
        tc_fence_before();
        cluster_arrive();
        cluster_wait();
        tc_fence_after();
        // an eighth of the rows: the parts in order, the scale, three terms
        const float scale = p.scales ? p.scales[T.x] : 1.0f;
        const uint32_t r0 = count * k / SC, r1 = count * (k + 1) / SC, quads = cols / 4;
        for (uint32_t i = t; i < (r1 - r0) * quads; i += TT) {
            const uint32_t r = r0 + i / quads, c = i % quads * 4;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (uint32_t q = 0; q < SC; ++q) {
                const float4 f = ld_cluster4(cluster_addr(part + r * pitch + c, q));
                v[0] += f.x;
                v[1] += f.y;
                v[2] += f.z;
                v[3] += f.w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = c + e < rank ? v[e] * scale : 0.0f;
            uint32_t lo[3], hi[3];
            terms2<3>(lo, v[0], v[1]);
            terms2<3>(hi, v[2], v[3]);
            uint16_t *dst = p.low + (uint64_t)(T.y + r) * 3 * cols_max + c;
#pragma unroll
            for (int j = 0; j < 3; ++j) *reinterpret_cast<uint2 *>(dst + j * cols_max) = make_uint2(lo[j], hi[j]);
        }
        cluster_arrive();   // parts may be written over once every CTA has read them
        cluster_wait();
    }
    __syncthreads();
    if (warp == 0) tmem_free(tmem, tmem_cols);
}

// ---------------------------------------------------------------- expand
constexpr uint32_t OM = 128;              // outputs of a tile

__host__ __device__ constexpr uint32_t kblocks(uint32_t max_rank) { return (round16(max_rank) + KB - 1) / KB; }
template <int NW> __host__ __device__ constexpr uint32_t expand_smem(uint32_t max_rank) {
    return 1024 + kblocks(max_rank) * PLANE * (3 + 2 * NW);
}

// Rows o0 .. o0 + 127 of B, 8 values (chunk t % 8 + 8 j) of rows t / 8 + 32 i.
struct BRegs {
    uint4 v[2][4];
};
__device__ __forceinline__ void load_b(BRegs &r, const LoraParams &p, const uint16_t *b, uint32_t rank, uint32_t o0) {
#pragma unroll
    for (uint32_t j = 0; j < 2; ++j) {
        const uint32_t c = threadIdx.x % 8 + 8 * j;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            const uint32_t o = o0 + threadIdx.x / 8 + 32 * i;
            r.v[j][i] = make_uint4(0, 0, 0, 0);
            if (c * 8 < rank && o < p.out_dim) r.v[j][i] = __ldg(reinterpret_cast<const uint4 *>(b + (uint64_t)o * p.max_rank + c * 8));
        }
    }
}
template <int NW> __device__ __forceinline__ void store_b(uint8_t *tile, uint32_t step, const BRegs &r, uint32_t rank) {
#pragma unroll
    for (uint32_t j = 0; j < 2; ++j) {
        const uint32_t c = threadIdx.x % 8 + 8 * j;
        if (c * 8 >= round16(rank)) continue;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            uint4 v = r.v[j][i];
            if (rank < c * 8 + 8) v = first_values(v, (int)rank - (int)c * 8);
            uint4 x[NW];
            if constexpr (NW == 2) terms_f16<NW>(x, v);
            else x[0] = v;
#pragma unroll
            for (int e = 0; e < NW; ++e)
                *reinterpret_cast<uint4 *>(tile + e * step + j * PLANE + swizzled(threadIdx.x / 8 + 32 * i, c % 8)) = x[e];
        }
    }
}

template <int NW> __global__ void __launch_bounds__(TT) k_lora_expand(const LoraParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    __shared__ uint64_t done[2];
    __shared__ uint32_t toks[TM];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t t = threadIdx.x, warp = t >> 5, lane = t & 31u;
    const uint32_t cols_max = round16(p.max_rank), kbs = kblocks(p.max_rank), step = kbs * PLANE;
    uint8_t *bs = smem + 3 * step;                           // two stages of NW terms
    if (t == 0) {
        mbar_init(&done[0], 1);
        mbar_init(&done[1], 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    grid_dep_wait();
    if (warp == 0) tmem_alloc(&tmem_slot, 2 * TM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t n_chunks = (p.out_dim + OM - 1) / OM;
    const uint64_t line = (uint64_t)p.tiles[0].x * n_chunks;
    uint64_t at = line * blockIdx.x / gridDim.x;
    const uint64_t end = line * (blockIdx.x + 1) / gridDim.x;
    uint32_t u = 0;                                          // chunks so far
    while (at < end) {
        const int4 T = p.tiles[1 + at / n_chunks];
        const uint32_t ch0 = (uint32_t)(at % n_chunks), ch1 = (uint32_t)min((uint64_t)n_chunks, ch0 + (end - at));
        at += ch1 - ch0;
        const uint32_t count = T.z, rank = T.w;
        __syncthreads();                                     // the last tile's tokens and terms are no longer read
        if (t < count) toks[t] = p.perm[T.y + t];
        if (T.x == NO_ADAPTER) {
            __syncthreads();
            const uint32_t o0 = ch0 * OM, wide = min(p.out_dim, ch1 * OM) - o0;
            for (uint32_t i = t; i < count * wide; i += 8 * TT) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t j = i + e * TT;
                    v[e] = p.base && j < count * wide ? p.base[(uint64_t)toks[j / wide] * p.base_stride + o0 + j % wide] : 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t j = i + e * TT;
                    if (j < count * wide) p.out[(uint64_t)toks[j / wide] * p.out_stride + o0 + j % wide] = v[e];
                }
            }
            continue;
        }
        const uint16_t *b = p.b + (uint64_t)T.x * p.b_stride;
        const uint32_t kr = round16(rank), cols = round16(count);
        const uint32_t idesc = tc_idesc(OM, cols, true);
        BRegs br;
        load_b(br, p, b, rank, ch0 * OM);
        for (uint32_t i = t; i < count * 3 * (kr / 8); i += TT) {
            const uint32_t c = i % (kr / 8), rj = i / (kr / 8), j = rj % 3, r = rj / 3;
            *reinterpret_cast<uint4 *>(smem + j * step + c / 8 * PLANE + swizzled(r, c % 8)) =
                *reinterpret_cast<const uint4 *>(p.low + ((uint64_t)(T.y + r) * 3 + j) * cols_max + c * 8);
        }
        // after a stage's stores: one accumulator, for a rank's few steps drop no more than roundings would
        const auto issue = [&](uint32_t v) {
            fence_async_smem();
            tc_fence_before();
            __syncthreads();
            if (warp == 0 && elect_one()) {
                tc_fence_after();
                for (uint32_t kb = 0; kb * KB < kr; ++kb)
                    issue_terms<3, NW, false>(tmem + (v & 1) * TM, 0, smem_addr(smem) + kb * PLANE, step,
                                              smem_addr(bs) + (v & 1) * NW * step + kb * PLANE, step, (int)(min(KB, kr - kb * KB) / 16), idesc,
                                              kb != 0, true);
                tc_commit(&done[v & 1]);
            }
        };
        store_b<NW>(bs + (u & 1) * NW * step, step, br, rank);
        issue(u);
        if (ch0 + 1 < ch1) load_b(br, p, b, rank, (ch0 + 1) * OM);
        for (uint32_t ch = ch0; ch < ch1; ++ch, ++u) {
            const uint32_t o = ch * OM + (warp & 3) * 32 + lane;
            const bool live = o < p.out_dim;
            const uint32_t c0 = (warp >> 2) * 16;
            float base[16];
            const auto load_base = [&](uint32_t c) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    base[e] = live && p.base && c + e < count ? p.base[(uint64_t)toks[c + e] * p.base_stride + o] : 0.0f;
            };
            if (c0 < cols) load_base(c0);
            tile_wait(&done[u & 1], (u / 2) & 1, p.err, &abort_flag);
            tc_fence_after();
            if (ch + 1 < ch1) {
                store_b<NW>(bs + ((u + 1) & 1) * NW * step, step, br, rank);
                issue(u + 1);
                if (ch + 2 < ch1) load_b(br, p, b, rank, (ch + 2) * OM);
            }
            for (uint32_t c = c0; c < cols; c += 32) {
                uint32_t d[16];
                tc_ld16(tmem + (u & 1) * TM + ((warp & 3) << 21) + c, d);
                tc_wait_ld();
                tc_regs_ready(d);
                float y[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = base[e] + __uint_as_float(d[e]);
                if (c + 32 < cols) load_base(c + 32);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (live && c + e < count) p.out[(uint64_t)toks[c + e] * p.out_stride + o] = y[e];
            }
        }
    }
    __syncthreads();
    if (warp == 0) tmem_free(tmem, 2 * TM);
}

// ---------------------------------------------------------------- launchers
template <int XK, int NX, int NW> cudaError_t launch_shrink(const LoraParams &p, unsigned clusters, cudaStream_t st) {
    static SmemAllowed allowed;
    const cudaError_t e = allow_smem(allowed, reinterpret_cast<const void *>(k_lora_shrink<XK, NX, NW>), shrink_smem<NX, NW>(LORA_MAX_RANK));
    if (e != cudaSuccess) return e;
    return launch_dependent(k_lora_shrink<XK, NX, NW>, p, dim3(clusters * SC), TT, shrink_smem<NX, NW>(p.max_rank), st);
}

template <int NW> cudaError_t launch_expand(const LoraParams &p, int num_sms, cudaStream_t st) {
    static SmemAllowed allowed;
    const cudaError_t e = allow_smem(allowed, reinterpret_cast<const void *>(k_lora_expand<NW>), expand_smem<NW>(LORA_MAX_RANK));
    if (e != cudaSuccess) return e;
    const uint32_t smem = expand_smem<NW>(p.max_rank);
    const unsigned ctas = (unsigned)num_sms * (smem <= 112 * 1024 ? 2 : 1);
    return launch_dependent(k_lora_expand<NW>, p, dim3(ctas), TT, smem, st);
}

// The most tiles that a call can have.
uint64_t most_tiles(uint64_t n_tok, uint64_t n_adapters) {
    return n_tok / TM + (n_tok < n_adapters + 1 ? n_tok : n_adapters + 1);
}
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

size_t lora_tc_scratch(uint32_t n_tok, uint32_t n_adapters, uint32_t max_rank) {
    return up256((1 + most_tiles(n_tok, n_adapters)) * sizeof(int4)) + up256((size_t)n_tok * 4) +
           (size_t)n_tok * 3 * round16(max_rank) * 2;
}

cudaError_t launch_lora_tc(const LoraParams &q, void *scratch, int num_sms, cudaStream_t st) {
    LoraParams p = q;
    uint8_t *at = static_cast<uint8_t *>(scratch);
    p.tiles = reinterpret_cast<int4 *>(at);
    at += up256((1 + most_tiles(p.n_tok, p.n_adapters)) * sizeof(int4));
    p.perm = reinterpret_cast<uint32_t *>(at);
    at += up256((size_t)p.n_tok * 4);
    p.low = reinterpret_cast<uint16_t *>(at);
    static SmemAllowed allowed;
    cudaError_t e = allow_smem(allowed, reinterpret_cast<const void *>(k_lora_route), (LORA_MAX_ADAPTERS + 1) * sizeof(int));
    if (e != cudaSuccess) return e;
    if ((e = launch_dependent(k_lora_route, p, dim3(1), RT, (p.n_adapters + 1) * sizeof(int), st)) != cudaSuccess) return e;
    const uint64_t most = most_tiles(p.n_tok, p.n_adapters), room = (uint64_t)num_sms * 2 / SC;
    const unsigned clusters = (unsigned)(most < room ? most : room);
    const bool bf = p.bf16;
    switch (p.x_type) {
        case Q8_TYPE_F32: e = bf ? launch_shrink<X_F32, 3, 1>(p, clusters, st) : launch_shrink<X_F32, 3, 2>(p, clusters, st); break;
        case Q8_TYPE_Q8_0: e = bf ? launch_shrink<X_Q8, 3, 1>(p, clusters, st) : launch_shrink<X_Q8, 3, 2>(p, clusters, st); break;
        case Q8_TYPE_BF16: e = bf ? launch_shrink<X_RAW, 1, 1>(p, clusters, st) : launch_shrink<X_RAW, 1, 2>(p, clusters, st); break;
        default: e = bf ? launch_shrink<X_F16, 2, 1>(p, clusters, st) : launch_shrink<X_RAW, 1, 1>(p, clusters, st);
    }
    if (e != cudaSuccess) return e;
    return bf ? launch_expand<1>(p, num_sms, st) : launch_expand<2>(p, num_sms, st);
}

}  // namespace q8
