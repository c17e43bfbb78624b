// q8_lora_tc.cu -- low-rank adapters of many tokens on the tensor cores: out[t] = base[t] + s_a B_a (A_a x[t]).
//
//   k_lora_route   one CTA orders the tokens by adapter and cuts them into tiles of up to 128 tokens of one adapter (or, where that
//                  spares something, groups of 4 for k_lora_groups in q8_lora.cu).  The order inside an adapter is left to
//                  chance: a token's result does not depend on its place in a tile or group.
//   k_lora_shrink  a cluster of 8 or 4 CTAs a tile, each a part of in_dim: low = A x with the tokens along the rows of the
//                  product.  The parts are added through distributed shared memory in a fixed order.
//   k_lora_expand  tiles of 128 outputs (rows) by the tile's tokens (columns): a warp's lanes hold neighbouring outputs of one
//                  token, so base and out are read and written in whole lines.
// 4096 tokens of 4 adapters, 4096 to 4096, rank 64, fp32 x: route 5 us, shrink 28 (67 MB of x: 1.3 us a
// K step of 32 KB on 128 SMs; with the terms, the products and the fence taken out 0.9, so the copies, the terms and their
// stores each take part), expand 26 (134 MB: 5.2 TB/s).  2048 tokens, 1024 to 32768, rank 16: expand 90 (537 MB, 6.0 TB/s).
//
// fp32 accuracy from 16-bit products: an fp32 value is the exact sum of three bf16 terms (8 of its 24 bits each), an fp16
// weight of two, and a product of two bf16 is exact in the fp32 accumulators.  Terms below 2^-24 of the
// product are left out.  The first terms' products and the rest are summed apart, or the rest first, for the tensor cores drop what
// is shifted out of a sum.  bf16 x takes one term, fp16 x two (one and kind f16 with fp16 adapters).
#include <atomic>
#include <cstring>

#include "q8_launch.h"
#include "q8_lora.cuh"
#include "q8_tcgen05.cuh"

namespace q8 {

bool encode_gather_tmap(CUtensorMap *map, const void *base, uint64_t cols, uint64_t rows, uint64_t row_stride, uint32_t size);
bool encode_rows32_tmap(CUtensorMap *map, const void *base, uint64_t cols, uint64_t rows, uint64_t row_stride);

namespace {

constexpr uint32_t TM = 128;              // tokens of a tile
constexpr uint32_t KB = 64;               // values of a K step: a 128-byte row of 16-bit terms
constexpr uint32_t PLANE = TM * 128;      // bytes of one term's 128 x 64 tile
constexpr uint32_t SC_MOST = 8;           // CTAs of a cluster of k_lora_shrink
constexpr uint32_t SMEM_MOST = 225 * 1024;   // dynamic shared memory; the barriers and token lists come on top
constexpr int NO_ADAPTER = -1;

// After an expired wait the warps go on (in bounds, on whatever the buffers hold) and may release a buffer whose copy has not landed.
// The flag is set before any such release, so a warp that reads it behind its own wait issues no copy then, and no barrier of a copy in
// flight is armed again.
__device__ __forceinline__ bool aborted(const volatile int *flag) { return __any_sync(0xffffffffu, *flag != 0); }
// Nothing lands after a CTA has gone, and no product is in flight when TMEM goes: a pause, by one warp that the others' end waits for.
// (Waits for the very copies and products, which have to be kept count of, took 0.5 us from every call; these take microseconds.)
__device__ __forceinline__ void linger(const volatile int *flag) {
    if (*flag == 0) return;
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000) {}
    __syncwarp();
}

// The next kernel's CTAs may come to free SMs and set themselves up (they wait for the end of this kernel before they read): 1.1 us
// a call in the two places.  They take TMEM only behind that wait: one that came early could take it from a kernel that this chain
// waits for.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------- route
constexpr int RT = 1024;

struct Sums {
    int tokens, tiles, groups;            // (where groups are weighed: adapters with enough tokens, tiles were all to have them, -)
    __device__ __forceinline__ Sums operator+(const Sums &o) const { return {tokens + o.tokens, tiles + o.tiles, groups + o.groups}; }
};
__device__ __forceinline__ Sums shfl_up(const Sums &s, int o) {
    return {__shfl_up_sync(0xffffffffu, s.tokens, o), __shfl_up_sync(0xffffffffu, s.tiles, o), __shfl_up_sync(0xffffffffu, s.groups, o)};
}
// Exclusive sums over the CTA; totals on every thread.
__device__ __forceinline__ Sums scan(const Sums &mine, Sums &total, Sums *warps) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    Sums s = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums v = shfl_up(s, o);
        if (lane >= o) s = s + v;
    }
    if (lane == 31) warps[w] = s;
    __syncthreads();
    if (w == 0) {
        Sums v = warps[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sums x = shfl_up(v, o);
            if (lane >= o) v = v + x;
        }
        warps[lane] = v;
    }
    __syncthreads();
    total = warps[31];
    if (w) s = s + warps[w - 1];
    return {s.tokens - mine.tokens, s.tiles - mine.tiles, s.groups - mine.groups};
}

constexpr int AT_ONCE = 4;                // tokens of a thread whose ids are loaded together

__global__ void __launch_bounds__(RT) k_lora_route(const LoraParams p) {
    extern __shared__ int counts[];       // [n_adapters + 1]: tokens (the last: of none), then the next free place
    __shared__ Sums warps[RT / 32];
    const int n = (int)p.n_adapters + 1, lane = threadIdx.x & 31;
    let_next_start();
    for (int i = threadIdx.x; i < n; i += RT) counts[i] = 0;
    grid_dep_wait();
    __syncthreads();
    const uint32_t rounds = (p.n_tok + AT_ONCE * RT - 1) / (AT_ONCE * RT);
    const int per = (n + RT - 1) / RT, b0 = min(n, (int)threadIdx.x * per), b1 = min(n, b0 + per);   // this thread's adapters
    const int32_t first_rank = b0 < n - 1 ? given_rank(p, b0) : 0;   // asked for with the ids
    const auto buckets = [&](uint32_t round, int (&b)[AT_ONCE], bool tell) {
#pragma unroll
        for (int q = 0; q < AT_ONCE; ++q) {
            const uint32_t i = (round * AT_ONCE + q) * RT + threadIdx.x;
            b[q] = i < p.n_tok ? p.adapter_of[i] : -2;
        }
#pragma unroll
        for (int q = 0; q < AT_ONCE; ++q) {
            if (b[q] == -2 && (round * AT_ONCE + q) * RT + threadIdx.x >= p.n_tok) {
                b[q] = -1;
            } else if (b[q] < 0 || b[q] >= n - 1) {
                if (tell && b[q] >= 0) raise_error(p.err, DEV_ERANGE);
                b[q] = n - 1;
            }
        }
    };
    int b[AT_ONCE];
    for (uint32_t r = 0; r < rounds; ++r) {
        buckets(r, b, true);
#pragma unroll
        for (int q = 0; q < AT_ONCE; ++q) {
            const unsigned same = __match_any_sync(0xffffffffu, b[q]);
            if (b[q] >= 0 && lane == __ffs(same) - 1) atomicAdd(&counts[b[q]], __popc(same));
        }
    }
    __syncthreads();
    // what becomes of an adapter's tokens: tiles, groups, or (no adapter, or one of rank 0) tiles that copy base
    Sums mine = {0, 0, 0}, total;
    // Groups spare a tile's work for few tokens, but are a kernel of their own: only where there are no tiles otherwise, or so
    // many that they would wait for each other
    bool groups = false;
    if (p.groups) {
        for (int i = b0; i < b1; ++i)
            if (i < n - 1 && counts[i]) mine = mine + Sums{counts[i] >= (int)LORA_TILE_MIN, (counts[i] + (int)TM - 1) / (int)TM, 0};
        scan(mine, total, warps);
        __syncthreads();
        groups = total.tokens == 0 || total.tiles > (int)LORA_TILES_AT_ONCE;
    }
    const auto kind = [&](int i, int c, int &rank, bool tell) -> Sums {
        rank = c && i < n - 1 ? (int)cut_rank(p, i == b0 ? first_rank : given_rank(p, i), tell) : 0;
        if (rank == 0) return {c, p.base == p.out ? 0 : (c + (int)TM - 1) / (int)TM, 0};
        if (groups && c < (int)LORA_TILE_MIN) return {c, 0, (c + (int)LORA_GROUP - 1) / (int)LORA_GROUP};
        return {c, (c + (int)TM - 1) / (int)TM, 0};
    };
    mine = {0, 0, 0};
    int rank;
    for (int i = b0; i < b1; ++i) mine = mine + kind(i, counts[i], rank, true);
    Sums at = scan(mine, total, warps);
    for (int i = b0; i < b1; ++i) {
        const int c = counts[i];
        const Sums k = kind(i, c, rank, false);
        counts[i] = at.tokens;
        for (int j = 0; j < k.tiles; ++j)
            p.tiles[1 + at.tiles + j] = make_int4(rank ? i : NO_ADAPTER, at.tokens + j * (int)TM, min((int)TM, c - j * (int)TM), rank);
        for (int j = 0; j < k.groups; ++j)
            p.groups[at.groups + j] = make_int4(i, at.tokens + j * (int)LORA_GROUP, min((int)LORA_GROUP, c - j * (int)LORA_GROUP), rank);
        at = at + k;
    }
    if (threadIdx.x == 0) p.tiles[0] = make_int4(total.tiles, total.groups, 0, 0);
    __syncthreads();
    for (uint32_t r = 0; r < rounds; ++r) {
        if (rounds > 1) buckets(r, b, false);
#pragma unroll
        for (int q = 0; q < AT_ONCE; ++q) {
            const unsigned same = __match_any_sync(0xffffffffu, b[q]);
            int place = 0;
            if (b[q] >= 0 && lane == __ffs(same) - 1) place = atomicAdd(&counts[b[q]], __popc(same));
            place = __shfl_sync(0xffffffffu, place, __ffs(same) - 1) + __popc(same & ((1u << lane) - 1u));
            if (b[q] >= 0) p.perm[place] = (r * AT_ONCE + q) * RT + threadIdx.x;
        }
    }
}

// ---------------------------------------------------------------- terms
// Two fp32 values as N packed bf16 pairs that sum to them: each takes the next 8 bits of what is left (three take all 24).
template <int N> __device__ __forceinline__ void terms2(uint32_t (&t)[N], float a, float b) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        t[i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
        if (i + 1 < N) {
            a = __fsub_rn(a, __uint_as_float(__float_as_uint(a) & 0xffff0000u));
            b = __fsub_rn(b, __uint_as_float(__float_as_uint(b) & 0xffff0000u));
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

// A tile's products over kr values (rows: the weights', columns: low's three terms), those that reach 2^-24, into one accumulator.
// The small ones come first: the tensor cores drop what is shifted out of a sum, so that only the steps of the first terms'
// products, one for 16 values, cost bits of the result.
template <int NW>
__device__ __forceinline__ void issue_terms(uint32_t d, uint32_t low, uint32_t w, uint32_t step, uint32_t kr, uint32_t idesc) {
    bool acc = false;
#pragma unroll
    for (int small = 2; small >= 0; --small)
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int i = small - j;
            if (i < 0) continue;
            for (uint32_t k = 0; k < kr; k += 16) {
                const uint32_t at = k / KB * PLANE;
                tc_mma_f16(d, sw128_desc(w + j * step + at) + k % KB / 8, sw128_desc(low + i * step + at) + k % KB / 8, idesc, acc);
                acc = true;
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

// Warps 0-15 turn raw rows into terms (x's in TMEM, the weights' in shared memory), two groups of eight a K step in turn, and
// finish the tile; warps 16-19 copy raw rows into a ring, warp 20 issues the products.
// The warps that fence their shared-memory writes for the tensor cores load nothing from global memory themselves: the fence
// waits for a warp's outstanding loads (with the loads in registers, two steps ahead, a step took 2.4 us).
constexpr int CONVERT = 512, GROUP = 256, COPY = 128, ST = CONVERT + COPY + 32;
constexpr uint32_t MAX_RAW = 6;

__host__ __device__ constexpr uint32_t round16(uint32_t r) { return (r + 15u) & ~15u; }

template <int XK> constexpr uint32_t RAW_PITCH = XK == X_F32 ? 256 : XK == X_Q8 ? 80 : 128;   // bytes of a raw row of x
struct ShrinkShape {
    uint32_t stage, raw, raws, body, smem;
};
template <int XK, int NW, bool RUNS> __host__ __device__ constexpr ShrinkShape shrink_shape(uint32_t max_rank) {
    ShrinkShape s{};
    const uint32_t cols = round16(max_rank), room = SMEM_MOST - 1024;
    s.stage = NW * cols * 128;                               // the weights' terms of a K step
    s.raw = TM * RAW_PITCH<XK> + cols * 128;
    s.body = 2 * s.stage;
    const uint32_t part = TM * (cols + (RUNS ? 0 : 4)) * 4;  // the CTA's sums take the stages' place, or (RUNS) lie behind them
    if (RUNS) s.body += part;
    else if (s.body < part) s.body = part;
    s.body = (s.body + 1023) & ~1023u;
    s.raws = (room - s.body) / s.raw;
    if (s.raws > MAX_RAW) s.raws = MAX_RAW;
    s.raws &= ~1u;                                           // a raw slot stays with one group, so none runs a phase of it ahead
    s.smem = 1024 + s.body + s.raws * s.raw;
    // Never two CTAs on an SM: each takes all of TMEM, and one that waits for it while its cluster waits for it could hold up a
    // cluster that the other CTA's cluster waits for.
    if (s.smem < 116 * 1024) s.smem = 116 * 1024;
    return s;
}
static_assert(shrink_shape<X_F32, 2, true>(LORA_MAX_RANK).raws == 2, "the largest: a slot of raw rows for each group");
// TMEM columns: the sums of the small terms' products, then up to four of the first terms' (the 16-value steps of a K step in turn:
// the tensor cores drop what is shifted out of a sum), from X_COLS on two stages of x
// terms (32 columns a term).
constexpr uint32_t X_COLS = 320, X_STAGE = 96;
__host__ __device__ constexpr uint32_t accumulators(uint32_t cols) { return cols <= 64 ? 4 : cols <= 96 ? 2 : 1; }
// What is dropped grows with a sum's length, by 2^-26 of the sum for every 16 values and always towards zero.  So long sums are taken in
// runs of 16 products an accumulator, and the runs added up in shared memory: 3e-7 whatever in_dim is, where 4096 values in one
// accumulator cost 4e-6 (and a plain fp32 product of 4096 to 32768 values 4 to 8e-7).  A run's end costs 0.5 to 0.8 us.
constexpr uint32_t RUN = 16;
__host__ __device__ constexpr uint32_t run_steps(uint32_t cols) { return RUN * accumulators(cols) / (KB / 16); }

// Place of 16-byte chunk c of row r in the CTA's sums: neighbouring rows' chunks lie in different banks.
template <bool RUNS> __device__ __forceinline__ uint32_t part_at(uint32_t r, uint32_t c, uint32_t cols) {
    if constexpr (RUNS) return r * cols + ((c ^ (cols & 16 ? r >> 1 & 3 : r & 7)) << 2);
    return r * (cols + 4) + c * 4;
}

// `bytes` of 16 or 4 global -> shared, the rest zeros.
__device__ __forceinline__ void cp_async16_part(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4_part(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// This thread's copies so far count as one arrival once they have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// An arrival at the same barrier of another CTA of the cluster, after all that this CTA's threads wrote before.
__device__ __forceinline__ void arrive_at(uint64_t *bar, uint32_t cta) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(bar, cta)) : "memory");
}
__device__ __forceinline__ bool cluster_bar_wait(uint64_t *bar, uint32_t parity, int *err, volatile int *abort, uint64_t limit_ns) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 0;; ++it) {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(smem_addr(bar)), "r"(parity)
                     : "memory");
        if (ok) return true;
        if ((it & 255u) == 255u) {
            if (*abort) return false;
            if (global_timer_ns() - t0 > limit_ns) {
                raise_error(err, DEV_ETIMEOUT);
                *abort = 1;
                return false;
            }
        }
    }
}

// Four rows' boxes, from column x on, global -> shared (counted on bar).
__device__ __forceinline__ void gather4(void *dst, const CUtensorMap *map, int x, const int (&r)[4], uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
            smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(smem_addr(bar))
        : "memory");
}
// One K step of x and of the weights, as they lie in memory, by the copying warps (thread b of 128).  fp32 rows lie in two tiles of
// 32 values, 16-bit ones in one of 64: 128 bytes a row, 16-byte chunks swizzled by row.  With x_tma four rows a time come through
// the copy engine (`full` counts them).
template <int XK>
__device__ __forceinline__ void copy_raw(const LoraParams &p, const CUtensorMap *tm_x, uint8_t *raw, const uint16_t *a, uint32_t rank,
                                         const uint32_t *toks, uint32_t count, uint32_t k0, uint32_t b, uint64_t *full) {
    const uint32_t x_dst = smem_addr(raw), w_dst = x_dst + TM * RAW_PITCH<XK>;
    const uint32_t left = min(KB, p.in_dim - k0);            // 32 or 64 values
    if constexpr (XK == X_Q8) {
        constexpr uint32_t WORDS = 18;                       // 68 bytes from an even address: the words that hold them
        const uint8_t *x = static_cast<const uint8_t *>(p.x);
#pragma unroll 6
        for (uint32_t i = b; i < count * WORDS; i += COPY) {
            const uint32_t row = i / WORDS, w = i - row * WORDS;
            const uint64_t s = ((uint64_t)toks[row] * (p.in_dim / QK) + k0 / QK) * QB, at = (s & ~(uint64_t)3) + 4 * w, end = s + left / QK * QB;
            cp_async4_part(x_dst + row * RAW_PITCH<XK> + 4 * w, x + (at < end ? at : 0), at < end ? (uint32_t)min((uint64_t)4, end - at) : 0u);
        }
        if (b == 0) mbar_arrive(full);
    } else if (p.x_tma) {
        constexpr uint32_t HALVES = XK == X_F32 ? 2 : 1;
        const uint32_t groups = (count + 3) / 4, halves = XK == X_F32 ? left / 32 : 1;
        if (b == 0) mbar_arrive_expect_tx(full, groups * halves * 512);
        const uint32_t g = b / 32 * 8 + b % 8, h = b % 32 / 8;
        if (h < HALVES && h < halves && g < groups) {
            int r[4];
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) r[j] = (int)toks[4 * g + j < count ? 4 * g + j : 0];
            gather4(raw + h * PLANE + g * 512, tm_x, (int)(k0 + 32 * h), r, full);
        }
        __syncwarp();
    } else {
        if (b == 0) mbar_arrive(full);
        constexpr uint32_t SIZE = XK == X_F32 ? 4 : 2, LANES = KB * SIZE / 16;   // threads of a row
        const uint32_t c = b % LANES;
        const bool in = c * 16 < left * SIZE;
        const uint8_t *x = static_cast<const uint8_t *>(p.x) + ((uint64_t)k0 * SIZE + (in ? c * 16 : 0));
#pragma unroll 8
        for (uint32_t row = b / LANES; row < count; row += COPY / LANES)
            cp_async16_part(x_dst + c / 8 * PLANE + swizzled(row, c % 8), x + (uint64_t)toks[row] * p.x_stride * SIZE, in ? 16 : 0);
    }
    const uint32_t c = b % 8;
    const bool in = c * 8 < left;
#pragma unroll 4
    for (uint32_t row = b / 8; row < rank; row += COPY / 8)
        cp_async16_part(w_dst + row * 128 + c * 16, a + (uint64_t)row * p.in_dim + k0 + (in ? c * 8 : 0), in ? 16 : 0);
}

// A raw step as terms (thread t of a group's 256): a thread has 32 of a row's 64 values, the row its lane of TMEM.
template <int XK, int NX, int NW>
__device__ __forceinline__ void convert(const LoraParams &p, uint32_t x_tmem, uint8_t *w_stage, const uint8_t *raw, const uint32_t *toks, uint32_t k0,
                                        uint32_t cols, uint32_t w_step, uint64_t *raw_empty, uint32_t t) {
    constexpr uint32_t WROWS = LORA_MAX_RANK * 8 / GROUP;
    const uint32_t row = t % 128, half = t / 128;
    uint4 x[8], w[WROWS];
    uint16_t d = 0;
    if constexpr (XK == X_Q8) {
        // the row's copy starts on a word; its first block 0 or 2 bytes behind that
        const uint32_t odd = ((uint32_t)(p.in_dim / QK) & toks[row] & 1u) * 2;
        const uint16_t *blk = reinterpret_cast<const uint16_t *>(raw + row * RAW_PITCH<XK> + odd + half * QB);
        const bool in = k0 + half * 32 < p.in_dim;
        d = in ? blk[0] : (uint16_t)0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t *q = reinterpret_cast<uint32_t *>(&x[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) q[e] = in ? blk[1 + 8 * i + 2 * e] | (uint32_t)blk[2 + 8 * i + 2 * e] << 16 : 0u;
        }
    } else {
        const bool in = k0 + half * 32 < p.in_dim;
#pragma unroll
        for (uint32_t i = 0; i < (XK == X_F32 ? 8u : 4u); ++i) {   // 16-byte pieces of 32 values
            x[i] = *reinterpret_cast<const uint4 *>(raw + (XK == X_F32 ? half * PLANE + swizzled(row, i) : swizzled(row, half * 4 + i)));
            if (!in) x[i] = make_uint4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < WROWS; ++i) {
        const uint32_t r = t / 8 + i * (GROUP / 8);
        if (r < cols) w[i] = *reinterpret_cast<const uint4 *>(raw + TM * RAW_PITCH<XK> + r * 128 + t % 8 * 16);
    }
    __syncwarp();
    if (t % 32 == 0) mbar_arrive(raw_empty);
    uint32_t terms[NX][16];                                  // pairs of values
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (XK == X_F32 || XK == X_Q8) {
            float v[4] = {__uint_as_float(x[i].x), __uint_as_float(x[i].y), __uint_as_float(x[i].z), __uint_as_float(x[i].w)};
            if constexpr (XK == X_Q8) {
                quants4(v, reinterpret_cast<const uint32_t *>(x)[i]);
                const float s = half_bits_to_float(d);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] *= s;
            }
            uint32_t lo[NX], hi[NX];
            terms2<NX>(lo, v[0], v[1]);
            terms2<NX>(hi, v[2], v[3]);
#pragma unroll
            for (int j = 0; j < NX; ++j) {
                terms[j][2 * i] = lo[j];
                terms[j][2 * i + 1] = hi[j];
            }
        } else if (i < 4) {
            uint4 y[NX];
            if constexpr (XK == X_F16) terms_f16<NX>(y, x[i]);
            else y[0] = x[i];
#pragma unroll
            for (int j = 0; j < NX; ++j) {
                terms[j][4 * i] = y[j].x;
                terms[j][4 * i + 1] = y[j].y;
                terms[j][4 * i + 2] = y[j].z;
                terms[j][4 * i + 3] = y[j].w;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NX; ++j) tc_st16(x_tmem + (row / 32 << 21) + j * 32 + half * 16, terms[j]);
#pragma unroll
    for (uint32_t i = 0; i < WROWS; ++i) {
        const uint32_t r = t / 8 + i * (GROUP / 8);
        if (r >= cols) continue;
        uint4 y[NW];
        if constexpr (NW == 2) terms_f16<NW>(y, w[i]);
        else y[0] = w[i];
#pragma unroll
        for (int j = 0; j < NW; ++j) *reinterpret_cast<uint4 *>(w_stage + j * w_step + swizzled(r, t % 8)) = y[j];
    }
    tc_wait_st();
    tc_fence_before();
}

// RUNS: sums of more than RUN products an accumulator are taken in runs.
template <int XK, int NX, int NW, bool RUNS>
__global__ void __launch_bounds__(ST, 1) k_lora_shrink(const LoraParams p, const __grid_constant__ CUtensorMap tm_x) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    __shared__ uint32_t toks[2][TM];
    __shared__ uint64_t raw_full[MAX_RAW], raw_empty[MAX_RAW], st_full[2], st_empty[2], tok_full[2], tok_empty[2], d_full, parts_ready,
        parts_read;
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const ShrinkShape sh = shrink_shape<XK, NW, RUNS>(p.max_rank);
    uint8_t *ring = smem + sh.body;
    const uint32_t t = threadIdx.x, warp = t >> 5, lane = t & 31u, k = cluster_rank(), SC = p.shrink_cluster;
    const uint32_t cols_max = round16(p.max_rank), w_step = cols_max * 128, turn = accumulators(cols_max) - 1;
    let_next_start();
    if (t == 0) {
        for (uint32_t i = 0; i < MAX_RAW; ++i) {
            mbar_init(&raw_full[i], COPY + 1);
            mbar_init(&raw_empty[i], GROUP / 32);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&st_full[i], GROUP / 32);
            mbar_init(&st_empty[i], 1);
            mbar_init(&tok_full[i], 1);
            mbar_init(&tok_empty[i], CONVERT / 32);
        }
        mbar_init(&d_full, 1);
        mbar_init(&parts_ready, SC);
        mbar_init(&parts_read, SC);
        abort_flag = 0;
        fence_mbar_init();
    }
    cluster_arrive();   // every CTA's barriers are there
    cluster_wait();
    grid_dep_wait();
    if (warp == ST / 32 - 1) tmem_alloc(&tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const int n_tiles = p.tiles[0].x, clusters = (int)(gridDim.x / SC);
    const uint32_t nb = (p.in_dim + KB - 1) / KB, kb0 = nb * k / SC, kb1 = nb * (k + 1) / SC;
    const uint32_t run = RUNS ? run_steps(cols_max) : 0xffffffffu;
    const uint64_t lim = wait_limit(p.wait_ns);
    const auto wait = [&](uint64_t *bar, uint32_t parity) { return tile_wait(bar, parity, p.err, &abort_flag, lim); };
    float *part = reinterpret_cast<float *>(smem + (RUNS ? 2 * sh.stage : 0));
    uint32_t n = 0, runs = 0;                                // K steps and (RUNS) runs so far
    int tiles = 0;                                           // tiles so far
    for (int tile = (int)(blockIdx.x / SC); tile < n_tiles; tile += clusters) {
        const int4 T = p.tiles[1 + tile];
        if (T.x == NO_ADAPTER) continue;
        const uint32_t count = T.z, rank = T.w, cols = round16(rank);
        uint32_t *tok = toks[tiles & 1];
        if (warp >= CONVERT / 32 && warp < (CONVERT + COPY) / 32) {
            // ------------------------------------------------ raw rows -> ring
            const uint32_t b = t - CONVERT;
            const uint16_t *a = p.a + (uint64_t)T.x * p.a_stride;
            if (tiles >= 2) wait(&tok_empty[tiles & 1], (tiles / 2 - 1) & 1);
            if (b < count) tok[b] = p.perm[T.y + b];
            named_bar_sync(1, COPY);
            if (b == 0) mbar_arrive(&tok_full[tiles & 1]);
            for (uint32_t kb = kb0; kb < kb1; ++kb, ++n) {
                const uint32_t r = n % sh.raws, use = n / sh.raws;
                if (use) wait(&raw_empty[r], (use - 1) & 1);
                if (p.withhold || aborted(&abort_flag)) continue;   // (withhold: the failure-detection test hook)
                copy_raw<XK>(p, &tm_x, ring + r * sh.raw, a, rank, tok, count, kb * KB, b, &raw_full[r]);
                cp_async_arrive(&raw_full[r]);
            }
        } else if (warp == ST / 32 - 1) {
            // ------------------------------------------------ products
            const uint32_t idesc = tc_idesc(TM, cols, !(XK == X_RAW && !p.bf16 && NW == 1));
            uint32_t of_run = 0;
            for (uint32_t kb = kb0; kb < kb1; ++kb, ++n) {
                const uint32_t s = n & 1;
                wait(&st_full[s], (n / 2) & 1);
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t x = tmem + X_COLS + s * X_STAGE, w = smem_addr(smem + s * sh.stage);
#pragma unroll
                    for (int i = 0; i < NX; ++i)
#pragma unroll
                        for (int j = 0; j < NW; ++j) {
                            if (i + j > 2) continue;
                            const bool small = i + j > 0, first_small = (i == 0 && j == 1) || (NW == 1 && i == 1);
                            const uint64_t wd = sw128_desc(w + j * w_step);
#pragma unroll
                            for (uint32_t k = 0; k < KB / 16; ++k) {
                                // the first product of an accumulator starts it
                                const bool starts = (!RUNS || small ? kb == kb0 : of_run == 0) && (small ? first_small && k == 0 : k <= turn);
                                tc_mma_f16_ta(small ? tmem : tmem + (1 + (k & turn)) * cols_max, x + i * 32 + k * 8, wd + 2 * k, idesc, !starts);
                            }
                        }
                    tc_commit(&st_empty[s]);
                    if (kb + 1 == kb1 || (RUNS && of_run + 1 == run)) tc_commit(&d_full);
                }
                __syncwarp();
                if (RUNS && ++of_run == run) of_run = 0;
            }
        } else {
            // ------------------------------------------------ terms
            wait(&tok_full[tiles & 1], (tiles / 2) & 1);
            const uint32_t row = (warp & 3) * 32 + lane;
            // this CTA's sums, one row a thread, from accumulator `first` on: stored, or (more) added to those of the runs before
            const auto take_sums = [&](uint32_t first, bool more) {
                for (uint32_t c = (warp >> 2) * 16; c < cols; c += 16 * (CONVERT / 128)) {
                    float sum[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum[e] = 0.0f;
                    if (kb0 < kb1)
                        for (uint32_t i = first; i <= 1 + turn; ++i) {
                            uint32_t d[16];
                            tc_ld16(tmem + ((warp & 3) << 21) + i * cols_max + c, d);
                            tc_wait_ld();
                            tc_regs_ready(d);
#pragma unroll
                            for (int e = 0; e < 16; ++e) sum[e] += __uint_as_float(d[e]);
                        }
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        float4 *at = reinterpret_cast<float4 *>(part + part_at<RUNS>(row, (c + e) / 4, cols));
                        float4 v = make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
                        if (RUNS && more) {
                            const float4 before = *at;
                            v = make_float4(before.x + v.x, before.y + v.y, before.z + v.z, before.w + v.w);
                        }
                        *at = v;
                    }
                }
                tc_fence_before();
            };
            uint32_t left = run;
            for (uint32_t kb = kb0; kb < kb1; ++kb, ++n) {
                const bool mine = n % 2 == t / GROUP;
                const uint32_t s = n & 1;
                if (mine) {
                    const uint32_t r = n % sh.raws, use = n / 2;
                    wait(&raw_full[r], (n / sh.raws) & 1);
                    if (use) wait(&st_empty[s], (use - 1) & 1);
                    tc_fence_after();
                    convert<XK, NX, NW>(p, tmem + X_COLS + s * X_STAGE, smem + s * sh.stage, ring + r * sh.raw, tok, kb * KB, cols, w_step,
                                        &raw_empty[r], t % GROUP);
                    fence_async_smem();
                    __syncwarp();
                }
                if constexpr (RUNS) {
                    // (the small terms' sums go on to the end: what they lose is small as well.)  The next run's first step is
                    // there, but released only once all have read
                    if (left-- == 0) {
                        wait(&d_full, runs++ & 1);
                        tc_fence_after();
                        take_sums(1, kb - kb0 > run);
                        named_bar_sync(2, CONVERT);
                        left = run - 1;
                    }
                }
                if (mine && lane == 0) mbar_arrive(&st_full[s]);
            }
            if (lane == 0) mbar_arrive(&tok_empty[tiles & 1]);
            if (kb0 < kb1) wait(&d_full, (RUNS ? runs++ : (uint32_t)tiles) & 1);
            tc_fence_after();
            named_bar_sync(2, CONVERT);
            take_sums(NX + NW > 2 ? 0 : 1, kb1 - kb0 > run);   // the small ones first
            named_bar_sync(2, CONVERT);
            if (t < SC) arrive_at(&parts_ready, t);
            cluster_bar_wait(&parts_ready, tiles & 1, p.err, &abort_flag, lim);
            // an eighth of the rows: the parts in order, the scale, three terms
            const float scale = p.scales ? p.scales[T.x] : 1.0f;
            const uint32_t r0 = count * k / SC, r1 = count * (k + 1) / SC, quads = cols / 4;
            for (uint32_t i = t; i < (r1 - r0) * quads; i += CONVERT) {
                const uint32_t r = r0 + i / quads, c = i % quads * 4;
                float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (uint32_t q = 0; q < SC_MOST; ++q) {
                    if (q >= SC) break;
                    const float4 f = ld_cluster4(cluster_addr(part + part_at<RUNS>(r, c / 4, cols), q));
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
            // the stages may be written over once every CTA has read
            named_bar_sync(2, CONVERT);
            if (t < SC) arrive_at(&parts_read, t);
            cluster_bar_wait(&parts_read, tiles & 1, p.err, &abort_flag, lim);
            tc_fence_after();
        }
        ++tiles;
    }
    if (warp >= CONVERT / 32 && warp < (CONVERT + COPY) / 32) cp_async_wait<0>();   // nothing lands after the CTA has gone
    tc_fence_before();
    __syncthreads();
    if (warp == ST / 32 - 1) {
        linger(&abort_flag);
        tmem_free(tmem, 512);
    }
    cluster_arrive();   // no CTA leaves while another may still read its sums, expired waits included
    cluster_wait();
}

// ---------------------------------------------------------------- expand
// base comes into a ring of slots of 32 tokens by 128 outputs (512-byte pieces of rows), the products are added in the slot or on
// the way out.  What is in flight does not depend on the registers of the warps that add.  With TMA (rows that start on 16-byte
// boundaries) the copy engine gathers and scatters the rows four at a time: through the load-store unit a slot's 16-byte copies
// and 4-byte stores took about as long as its bytes take from memory (4096 x 4096 outputs: 36 us).
//   warps 0-15   four groups of four, slots in turn: slot + product -> out
//   warps 16-17  base -> slots, in turn
//   warp 18      products
//   warps 19-22  B (and at a new tile the rank-sized sums) -> shared memory
constexpr uint32_t OM = 128;              // outputs of a tile
constexpr int E_GROUPS = 4, E_COPY0 = 4 * E_GROUPS, E_COPIES = 2, E_MMA = E_COPY0 + E_COPIES, E_B0 = E_MMA + 1, B_THREADS = 128, ET = E_B0 * 32 + B_THREADS;
constexpr uint32_t SLOT_TOK = 32, SLOT = SLOT_TOK * OM * 4, MAX_SLOTS = 8;

__host__ __device__ constexpr uint32_t kblocks(uint32_t max_rank) { return (round16(max_rank) + KB - 1) / KB; }
struct ExpandShape {
    uint32_t kbs, b_stages, slots, smem;
};
template <int NW> __host__ __device__ constexpr ExpandShape expand_shape(uint32_t max_rank) {
    ExpandShape s{};
    s.kbs = kblocks(max_rank);
    s.b_stages = NW * s.kbs > 2 ? 1 : 2;
    const uint32_t fixed = 1024 + s.kbs * PLANE * (3 + NW * s.b_stages), room = SMEM_MOST - fixed;
    // a multiple of the groups: a slot stays with one group and one copying warp, so none runs a phase of it ahead
    s.slots = room / SLOT < MAX_SLOTS ? room / SLOT & ~3u : MAX_SLOTS;
    s.smem = fixed + s.slots * SLOT;
    return s;
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }

// A CTA's share of the line of (tile, 128 outputs), one after another.
struct Units {
    uint64_t at, end;
    uint32_t n_chunks, tile, chunk;
    int4 T;                               // {adapter, first of perm, tokens, rank}
    bool new_tile;
    __device__ __forceinline__ Units(const LoraParams &p) {
        n_chunks = (p.out_dim + OM - 1) / OM;
        const uint64_t line = (uint64_t)p.tiles[0].x * n_chunks;
        at = line * blockIdx.x / gridDim.x;
        end = line * (blockIdx.x + 1) / gridDim.x;
        if (at < end) first(p);
    }
    __device__ __forceinline__ void first(const LoraParams &p) {
        tile = (uint32_t)(at / n_chunks);
        chunk = (uint32_t)(at % n_chunks);
        T = p.tiles[1 + tile];
        new_tile = true;
    }
    __device__ __forceinline__ bool live() const { return at < end; }
    __device__ __forceinline__ void next(const LoraParams &p) {
        new_tile = false;
        if (++at >= end) return;
        if (++chunk == n_chunks) {
            chunk = 0;
            T = p.tiles[1 + ++tile];
            new_tile = true;
        }
    }
};

__device__ __forceinline__ void scatter4(const CUtensorMap *map, int x, const int (&r)[4], const void *src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile::scatter4.bulk_group [%0, {%1, %2, %3, %4, %5}], [%6];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(smem_addr(src))
                 : "memory");
}
// Rows 4 lane .. 4 lane + 3 of a slot's tokens (lane l holds token l).
__device__ __forceinline__ void four_rows(int (&r)[4], uint32_t tok) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = (int)__shfl_sync(0xffffffffu, tok, (4 * lane + j) & 31);
}

// TMA: rows of base and out start on 16-byte boundaries and have whole 16 bytes; tm_base, tm_out: their maps.
template <int NW, bool TMA>
__global__ void __launch_bounds__(ET, 1) k_lora_expand(const LoraParams p, const __grid_constant__ CUtensorMap tm_base,
                                                       const __grid_constant__ CUtensorMap tm_out) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    __shared__ uint64_t full[MAX_SLOTS], empty[MAX_SLOTS], b_full[2], b_empty[2], d_full[2], d_empty[2];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t t = threadIdx.x, warp = t >> 5, lane = t & 31u;
    const ExpandShape sh = expand_shape<NW>(p.max_rank);
    const uint32_t cols_max = round16(p.max_rank), step = sh.kbs * PLANE;
    uint8_t *bs = smem + 3 * step, *ring = bs + sh.b_stages * NW * step;
    if (t == 0) {
        if (TMA) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_base)) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_out)) : "memory");
        }
        for (uint32_t i = 0; i < MAX_SLOTS; ++i) {
            mbar_init(&full[i], 32);
            mbar_init(&empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b_full[i], B_THREADS);
            mbar_init(&b_empty[i], 1);
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], 4 * E_GROUPS);
        }
        abort_flag = 0;
        fence_mbar_init();
    }
    grid_dep_wait();
    if (warp == E_MMA) tmem_alloc(&tmem_slot, 2 * TM);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint64_t lim = wait_limit(p.wait_ns);
    const auto wait = [&](uint64_t *bar, uint32_t parity) { return tile_wait(bar, parity, p.err, &abort_flag, lim); };
    if (warp < E_COPY0) {
        const uint32_t group = warp >> 2, q = warp & 3, col = q * 32 + lane, out_step = (uint32_t)p.out_stride * 4;
        uint32_t n = 0, u = 0;                               // slots and products so far
        int sent = -1;                                       // the slot that the copy engine may still read (warp q = 0)
        const auto release_sent = [&] {
            if (sent < 0) return;
            bulk_wait_read<0>();
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[sent]);
            sent = -1;
        };
        for (Units w(p); w.live(); w.next(p)) {
            const uint32_t count = w.T.z, o = w.chunk * OM + col;
            const bool product = w.T.x != NO_ADAPTER;
            const bool all = w.chunk * OM + OM <= p.out_dim;
            uint8_t *const to = reinterpret_cast<uint8_t *>(p.out + o);
            bool ready = !product;
            for (uint32_t s0 = 0; s0 < count; s0 += SLOT_TOK, ++n) {
                if (n % E_GROUPS != group) continue;
                if (TMA) release_sent();
                const uint32_t slot = n % sh.slots, rows = min(SLOT_TOK, count - s0);
                const uint32_t sent_rows = TMA && all ? rows & ~3u : 0;   // rows that leave from the slot; the others from here
                float *f = reinterpret_cast<float *>(ring + slot * SLOT) + col;
                const uint32_t tok = lane < rows ? p.perm[w.T.y + s0 + lane] : 0;
                if (!ready) {
                    wait(&d_full[u & 1], (u / 2) & 1);
                    tc_fence_after();
                    ready = true;
                }
                wait(&full[slot], (n / sh.slots) & 1);
                if (product || !p.base || sent_rows < rows) {   // else the slot leaves as it came
#pragma unroll
                    for (uint32_t h = 0; h < SLOT_TOK; h += 16) {
                        if (h >= rows) break;
                        uint32_t d[16];
                        float y[16];
                        if (product) tc_ld16(tmem + (u & 1) * TM + (q << 21) + s0 + h, d);
#pragma unroll
                        for (uint32_t e = 0; e < 16; ++e) y[e] = p.base ? f[(h + e) * OM] : 0.0f;
                        if (product) {
                            tc_wait_ld();
                            tc_regs_ready(d);
#pragma unroll
                            for (int e = 0; e < 16; ++e) y[e] += __uint_as_float(d[e]);
                        }
                        if (sent_rows >= h + 16) {
#pragma unroll
                            for (uint32_t e = 0; e < 16; ++e) f[(h + e) * OM] = y[e];
                        } else if (all && rows == SLOT_TOK) {
#pragma unroll
                            for (uint32_t e = 0; e < 16; ++e)
                                *reinterpret_cast<float *>(to + (uint64_t)__shfl_sync(0xffffffffu, tok, h + e) * out_step) = y[e];
                        } else {
#pragma unroll
                            for (uint32_t e = 0; e < 16; ++e) {
                                const uint32_t row = __shfl_sync(0xffffffffu, tok, h + e);
                                if (h + e < sent_rows) f[(h + e) * OM] = y[e];
                                else if (h + e < rows && o < p.out_dim) *reinterpret_cast<float *>(to + (uint64_t)row * out_step) = y[e];
                            }
                        }
                    }
                }
                if (sent_rows) {
                    fence_async_smem();
                    named_bar_sync(1 + (int)group, 128);
                    if (q == 0) {
                        int r[4];
                        four_rows(r, tok);
                        if (lane * 4 < sent_rows) scatter4(&tm_out, (int)(w.chunk * OM), r, ring + slot * SLOT + lane * 4 * OM * 4);
                        bulk_commit();
                        sent = (int)slot;
                        // with one slot a group its next one waits for this
                        if (sh.slots < 2 * E_GROUPS) release_sent();
                    }
                }
                if (!sent_rows || q != 0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[slot]);
                }
            }
            if (product) {
                if (!ready) wait(&d_full[u & 1], (u / 2) & 1);   // a tile of few slots is the other groups' alone
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&d_empty[u & 1]);
                ++u;
            }
        }
        if (TMA) release_sent();
    } else if (warp < E_COPY0 + E_COPIES) {
        uint32_t n = 0;                                      // slots so far
        for (Units w(p); w.live(); w.next(p)) {
            const uint32_t count = w.T.z, o0 = w.chunk * OM, width = min(OM, p.out_dim - o0);
            for (uint32_t s0 = 0; s0 < count; s0 += SLOT_TOK, ++n) {
                if (n % E_COPIES != warp - E_COPY0) continue;
                const uint32_t slot = n % sh.slots, rows = min(SLOT_TOK, count - s0), uses = n / sh.slots;
                const uint32_t tok = p.base && lane < rows ? p.perm[w.T.y + s0 + lane] : 0;
                if (uses) wait(&empty[slot], (uses - 1) & 1);
                if (aborted(&abort_flag) || (p.withhold && warp > E_COPY0)) continue;   // (withhold: the failure-detection test hook)
                if (TMA && p.base && width == OM) {
                    // whole groups of four rows; a last group reads some row again
                    const uint32_t first = __shfl_sync(0xffffffffu, tok, 0);
                    int r[4];
                    four_rows(r, lane < rows ? tok : first);
                    const uint32_t groups = (rows + 3) / 4;
                    if (lane == 0) mbar_arrive_expect_tx(&full[slot], groups * 4 * OM * 4);
                    else mbar_arrive(&full[slot]);
                    __syncwarp();
                    if (lane < groups) gather4(ring + slot * SLOT + lane * 4 * OM * 4, &tm_base, (int)o0, r, &full[slot]);
                    continue;
                }
                if (p.base) {
                    const uint32_t dst = smem_addr(ring + slot * SLOT);
                    const float *base = p.base + o0;
                    const uint32_t base_step = (uint32_t)p.base_stride * 4;
#pragma unroll 8
                    for (uint32_t e = 0; e < rows; ++e) {
                        const float *src = reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(base) +
                                                                           (uint64_t)__shfl_sync(0xffffffffu, tok, e) * base_step);
                        if constexpr (TMA) {
                            if (lane * 4 < width) cp_async16_part(dst + e * OM * 4 + lane * 16, src + lane * 4, 16);
                        } else {
#pragma unroll
                            for (uint32_t c = lane; c < OM; c += 32)
                                if (c < width) cp_async4_part(dst + e * OM * 4 + c * 4, src + c, 4);
                        }
                    }
                }
                cp_async_arrive(&full[slot]);
            }
        }
        cp_async_wait<0>();                                  // nothing lands after the CTA has gone
    } else if (warp == E_MMA) {
        uint32_t u = 0;
        for (Units w(p); w.live(); w.next(p)) {
            if (w.T.x == NO_ADAPTER) continue;
            const uint32_t kr = round16(w.T.w), st = u % sh.b_stages;
            const uint32_t idesc = tc_idesc(OM, round16(w.T.z), true);
            wait(&b_full[st], (u / sh.b_stages) & 1);
            if (u >= 2) wait(&d_empty[u & 1], (u / 2 - 1) & 1);
            tc_fence_after();
            if (elect_one()) {
                issue_terms<NW>(tmem + (u & 1) * TM, smem_addr(smem), smem_addr(bs) + st * NW * step, step, kr, idesc);
                tc_commit(&b_empty[st]);
                tc_commit(&d_full[u & 1]);
            }
            __syncwarp();
            ++u;
        }
    } else {
        const uint32_t b = t - E_B0 * 32;
        uint32_t u = 0;
        for (Units w(p); w.live(); w.next(p)) {
            if (w.T.x == NO_ADAPTER) continue;
            const uint32_t rank = w.T.w, kr = round16(rank), st = u % sh.b_stages, o0 = w.chunk * OM;
            const uint16_t *wb = p.b + (uint64_t)w.T.x * p.b_stride;
            uint4 v[8];
            const auto load = [&](uint32_t c) {
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) {
                    const uint32_t o = o0 + b / 8 + 16 * i;
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (c * 8 < rank && o < p.out_dim) v[i] = __ldg(reinterpret_cast<const uint4 *>(wb + (uint64_t)o * p.max_rank + c * 8));
                }
            };
            load(b % 8);
            if (u >= sh.b_stages) wait(&b_empty[st], (u / sh.b_stages - 1) & 1);
            if (w.new_tile || u == 0) {
                // the sums of the tile before are read until its last product is done
                if (u) wait(&b_empty[(u - 1) % sh.b_stages], ((u - 1) / sh.b_stages) & 1);
                const uint32_t row_chunks = kr / 8;
#pragma unroll 4
                for (uint32_t i = b; i < (uint32_t)w.T.z * 3 * row_chunks; i += B_THREADS) {
                    const uint32_t c = i % row_chunks, rj = i / row_chunks, j = rj % 3, r = rj / 3;
                    cp_async16(smem_addr(smem + j * step + c / 8 * PLANE + swizzled(r, c % 8)),
                               p.low + ((uint64_t)(w.T.y + r) * 3 + j) * cols_max + c * 8, true);
                }
                cp_async_commit();
                cp_async_wait<0>();
            }
            for (uint32_t c = b % 8;; c += 8) {
                if (c * 8 < kr) {
#pragma unroll
                    for (uint32_t i = 0; i < 8; ++i) {
                        uint4 x[NW], y = v[i];
                        if (rank < c * 8 + 8) y = first_values(y, (int)rank - (int)c * 8);
                        if constexpr (NW == 2) terms_f16<NW>(x, y);
                        else x[0] = y;
#pragma unroll
                        for (int e = 0; e < NW; ++e)
                            *reinterpret_cast<uint4 *>(bs + (st * NW + e) * step + c / 8 * PLANE + swizzled(b / 8 + 16 * i, c % 8)) = x[e];
                    }
                }
                if ((c + 8) / 8 * KB >= kr) break;
                load(c + 8);
            }
            fence_async_smem();
            mbar_arrive(&b_full[st]);
            ++u;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == E_MMA) {
        linger(&abort_flag);
        tmem_free(tmem, 2 * TM);
    }
}

// ---------------------------------------------------------------- launchers
template <int XK, int NX, int NW, bool RUNS> cudaError_t launch_shrink_of(LoraParams p, unsigned tiles, int num_sms, cudaStream_t st) {
    static SmemAllowed allowed;
    const auto kernel = k_lora_shrink<XK, NX, NW, RUNS>;
    cudaError_t e = allow_smem(allowed, reinterpret_cast<const void *>(kernel), SMEM_MOST);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(ST);
    cfg.dynamicSmemBytes = shrink_shape<XK, NW, RUNS>(p.max_rank).smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    // Clusters that fit at a time are fewer than SMs / CTAs (15 of 8, 36 of 4 on 152 SMs): more tiles than clusters of 8
    // take clusters of 4 (4096 tokens with clusters of 8: three rounds, 52 us; of 4: one, 31).  Ranks above 96, whose runs are a quarter
    // as long, do so from two rounds on (4096 to 4096, rank 128, whole calls: 36 tiles 92 and 67 us; 8192 inputs, 12 tiles of at most 16:
    // 49 and 69).
    const unsigned most_rounds = accumulators(round16(p.max_rank)) > 1 ? 1 : 2;
    int dev = -1, fit = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    static std::atomic<int> fits[2][64];                     // clusters of 8 and of 4 that fit on a device, asked for once
    for (p.shrink_cluster = SC_MOST;; p.shrink_cluster /= 2) {
        std::atomic<int> *known = dev >= 0 && dev < 64 ? &fits[p.shrink_cluster == 4][dev] : nullptr;
        attr[1].val.clusterDim.x = p.shrink_cluster;
        fit = known ? known->load(std::memory_order_relaxed) : 0;
        if (fit < 1) {
            cfg.gridDim = dim3((unsigned)num_sms / p.shrink_cluster * p.shrink_cluster);
            if ((e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg)) != cudaSuccess) return e;
            if (fit < 1) fit = 1;
            if (known) known->store(fit, std::memory_order_relaxed);
        }
        if (tiles <= most_rounds * (unsigned)fit || p.shrink_cluster == 4) break;
    }
    // the kernel of whole sums takes no more K steps a CTA than one run has
    const uint32_t steps = ((p.in_dim + KB - 1) / KB + p.shrink_cluster - 1) / p.shrink_cluster;
    if constexpr (!RUNS)
        if (steps > run_steps(round16(p.max_rank))) return launch_shrink_of<XK, NX, NW, true>(p, tiles, num_sms, st);
    cfg.gridDim = dim3((tiles < (unsigned)fit ? tiles : (unsigned)fit) * p.shrink_cluster);
    CUtensorMap x;
    memset(&x, 0, sizeof x);
    p.x_tma = XK != X_Q8 && encode_gather_tmap(&x, p.x, p.in_dim, p.n_tok, p.x_stride, XK == X_F32 ? 4 : 2);
    e = cudaLaunchKernelEx(&cfg, kernel, (const LoraParams)p, (const CUtensorMap)x);
    return e == cudaSuccess ? cudaGetLastError() : e;
}
template <int XK, int NX, int NW> cudaError_t launch_shrink(const LoraParams &p, unsigned tiles, int num_sms, cudaStream_t st) {
    return launch_shrink_of<XK, NX, NW, false>(p, tiles, num_sms, st);
}

template <int NW, bool TMA>
cudaError_t launch_expand_rows(const LoraParams &p, const CUtensorMap &tm_base, const CUtensorMap &tm_out, int num_sms, cudaStream_t st) {
    static SmemAllowed allowed;
    cudaError_t e = allow_smem(allowed, reinterpret_cast<const void *>(k_lora_expand<NW, TMA>), SMEM_MOST);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)num_sms);
    cfg.blockDim = dim3(ET);
    cfg.dynamicSmemBytes = expand_shape<NW>(p.max_rank).smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_lora_expand<NW, TMA>, p, tm_base, tm_out);
    return e == cudaSuccess ? cudaGetLastError() : e;
}
template <int NW> cudaError_t launch_expand(const LoraParams &p, int num_sms, cudaStream_t st) {
    CUtensorMap base, out;
    if (p.out_dim % 4 == 0 && encode_rows32_tmap(&out, p.out, p.out_dim, p.n_tok, p.out_stride) &&
        encode_rows32_tmap(&base, p.base ? p.base : p.out, p.out_dim, p.n_tok, p.base ? p.base_stride : p.out_stride))
        return launch_expand_rows<NW, true>(p, base, out, num_sms, st);
    memset(&base, 0, sizeof base);
    return launch_expand_rows<NW, false>(p, base, base, num_sms, st);
}

// The most tiles that a call can have: c tokens take (c - 1) / TM + 1, of as many adapters (or none) as there may be.
uint64_t most_tiles(uint64_t n_tok, uint64_t n_adapters) {
    const uint64_t shares = n_tok < n_adapters + 1 ? n_tok : n_adapters + 1;
    return (n_tok - shares) / TM + shares;
}
uint64_t most_groups(uint64_t n_tok, uint64_t n_adapters) {
    const uint64_t few = n_adapters * ((LORA_TILE_MIN + LORA_GROUP - 2) / LORA_GROUP);
    return n_tok < few ? n_tok : few;
}
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
size_t list_bytes(const uint64_t n) { return up256(n * sizeof(int4)); }

}  // namespace

size_t lora_tc_scratch(uint32_t n_tok, uint32_t n_adapters, uint32_t max_rank) {
    return list_bytes(1 + most_tiles(n_tok, n_adapters)) + list_bytes(most_groups(n_tok, n_adapters)) + up256((size_t)n_tok * 4) +
           (size_t)n_tok * 3 * round16(max_rank) * 2;
}

cudaError_t launch_lora_tc(const LoraParams &q, void *scratch, int num_sms, cudaStream_t st) {
    LoraParams p = q;
    uint8_t *at = static_cast<uint8_t *>(scratch);
    p.tiles = reinterpret_cast<int4 *>(at);
    at += list_bytes(1 + most_tiles(p.n_tok, p.n_adapters));
    // Where all tiles run at once in any case there are no groups, and no kernel for them (333 tokens of 12 adapters: 24.0 us, 26.3
    // with it).
    const bool groups = most_tiles(p.n_tok, p.n_adapters) > LORA_TILES_AT_ONCE;
    p.groups = groups ? reinterpret_cast<int4 *>(at) : nullptr;
    at += list_bytes(most_groups(p.n_tok, p.n_adapters));
    p.perm = reinterpret_cast<uint32_t *>(at);
    at += up256((size_t)p.n_tok * 4);
    p.low = reinterpret_cast<uint16_t *>(at);
    static SmemAllowed allowed;
    cudaError_t e = allow_smem(allowed, reinterpret_cast<const void *>(k_lora_route), (LORA_MAX_ADAPTERS + 1) * sizeof(int));
    if (e != cudaSuccess) return e;
    if ((e = launch_dependent(k_lora_route, p, dim3(1), RT, (p.n_adapters + 1) * sizeof(int), st)) != cudaSuccess) return e;
    if (groups && (e = launch_lora_groups(p, num_sms, st)) != cudaSuccess) return e;
    const uint64_t most = most_tiles(p.n_tok, p.n_adapters);
    const unsigned tiles = (unsigned)(most < 65536 ? most : 65536);
    const bool bf = p.bf16;
    switch (p.x_type) {
        case Q8_TYPE_F32: e = bf ? launch_shrink<X_F32, 3, 1>(p, tiles, num_sms, st) : launch_shrink<X_F32, 3, 2>(p, tiles, num_sms, st); break;
        case Q8_TYPE_Q8_0: e = bf ? launch_shrink<X_Q8, 3, 1>(p, tiles, num_sms, st) : launch_shrink<X_Q8, 3, 2>(p, tiles, num_sms, st); break;
        case Q8_TYPE_BF16: e = bf ? launch_shrink<X_RAW, 1, 1>(p, tiles, num_sms, st) : launch_shrink<X_RAW, 1, 2>(p, tiles, num_sms, st); break;
        default: e = bf ? launch_shrink<X_F16, 2, 1>(p, tiles, num_sms, st) : launch_shrink<X_RAW, 1, 1>(p, tiles, num_sms, st);
    }
    if (e != cudaSuccess) return e;
    return bf ? launch_expand<1>(p, num_sms, st) : launch_expand<2>(p, num_sms, st);
}

}  // namespace q8
