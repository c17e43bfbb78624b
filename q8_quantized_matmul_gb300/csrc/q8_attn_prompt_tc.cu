// q8_attn_prompt_tc.cu -- attention over whole packed prompts on the 5th-generation tensor cores,
// heads of 128 values.
//
// A CTA works on 256 rows as two tiles of 128, over key tiles of 128.  A row is a query of one head; the heads
// of a group may be packed beside each other (attn_prompt_pack), so short prompts fill their tiles too.  Per key
// tile and query tile: S = Q K^T (8 UMMAs) into 128 TMEM columns; one thread per row reads its S,
// keeps the running maximum m and sum l, writes P = 2^(S - m) as 16-bit pairs over S; O += P V
// (8 UMMAs, P from TMEM) into 128 further columns.  S of both tiles (256 columns) and O of both fill
// the SM's 512 columns.  While the threads of one tile work on its softmax the tensor cores run the
// other tile's products, so the two overlap: a key tile costs the tensor pipe about 2048
// cycles for both query tiles and the softmax warps about 1350.  One prompt of 8192 tokens with 32 heads on 8 takes
// 339 us (1.62 PFLOP/s, at the card's power limit), one of 4096 tokens 101 us (1.36).
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since the last time (the weights
// then stay below 2^8 in bf16; in fp16 they are counted in units 2^7 smaller, see weight_ref, and stay below 2^15);
// the result is the same sum in other units.  The
// threads of a tile do that themselves: S of the next key tile is complete only after this tile's P V is,
// so O is at rest between the two.
//
// Warps: 0-3 and 4-7 the softmax of the two tiles (thread = row = TMEM lane), 8 the TMA producer, 9 the
// UMMA issuer, 10-11 the V guard.  The guard holds every V tile until it has removed values that are not
// finite from tiles that some rows may not see (0 times infinity would reach them); they are added at the
// end to the rows that do see them (prompt_restore).
//
// Calls with more tiles than SMs run one persistent CTA per SM over a list of tiles, longest first, that a
// small kernel writes: the loads and the first S of a CTA's next tile then run under the last softmax and the
// stores of this one (separate CTAs spent 9300 cycles each before the first and after the last product).
// Smaller calls give each CTA its one tile directly and save that launch.
//
// Every wait is bounded; after one expires nothing more is issued and copies in flight are drained.
#include "q8_attn.cuh"
#include "q8_attn_prompt_tc.cuh"
#include "q8_kv.h"
#include "q8_launch.h"

namespace q8 {

bool encode_rows16_tmap(CUtensorMap *map, const void *base, uint64_t cols, uint64_t rows, uint64_t row_stride,
                        uint32_t box_rows, bool bf16);
bool encode_3d16_tmap(CUtensorMap *map, const void *base, uint64_t cols, uint64_t n1, uint64_t n2, uint64_t stride1,
                      uint64_t stride2, uint32_t box1, uint32_t box2, bool bf16);

namespace {

struct Pt {
    static constexpr int D = 128, BN = 128;
    static constexpr int CH = 2;                             // 64-value chunks of a row, 16 KB a chunk of 128 rows
    static constexpr int TILE = 128 * D * 2;
    // stage u holds the values of key tile u - 1 and the keys of tile u, which are used in one go
    static constexpr int STAGE = 2 * TILE;
    static constexpr int NST = 2;
    static constexpr int THREADS = 384;
    static constexpr int NBAR = 2 + 3 * NST + 2 + 2 + 2 + 1;
    static constexpr int SMEM = 1024 + 2 * TILE + NST * STAGE + NBAR * 8 + 128;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// ---------------------------------------------------------------- list of tiles
constexpr int LIST_THREADS = 1024, LIST_BINS = 1024;

__device__ __forceinline__ int tile_cost(const PromptTile &w, uint32_t window) {
    const int last = w.last(w.rows - 1);
    return last < 0 ? 0 : last / 128 + 1 - w.first(0, window) / 128;
}

// One CTA: all tiles of tile_tokens queries, the ones with the most key tiles first (counting sort; the order
// among equals does not matter to any result).
__global__ void __launch_bounds__(LIST_THREADS) k_attn_prompt_list(const AttnPromptParams p) {
    __shared__ int bin[LIST_BINS];
    __shared__ int wsum[32];
    __shared__ uint32_t wrows[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_wait();
    const int32_t *ks = p.k_start ? p.k_start : p.q_start;
    bin[tid] = 0;
    __syncthreads();
    PromptTile *list = reinterpret_cast<PromptTile *>(p.list + 1);
    // a lane per sequence; the warp together for long ones, a lane per tile; go: whether to, given a lane's rows
    auto each = [&](auto go, auto f) {
        const uint32_t per = min(32u, (p.n_seq + 31) / 32);   // sequences of a warp: few ones are spread over the warps
        for (uint32_t s0 = warp * per; s0 < p.n_seq; s0 += 32 * per) {
            const uint32_t s = s0 + lane;
            int qa = 0, qe = 0, ka = 0, ke = 0;
            if (lane < per && s < p.n_seq) {
                const int4 raw = make_int4(p.q_start[s], p.q_start[s + 1], ks[s], ks[s + 1]);
                qa = prompt_bound(raw.x, p.n_q);
                qe = prompt_bound(raw.y, p.n_q);
                ka = prompt_bound(raw.z, p.n_k);
                ke = prompt_bound(raw.w, p.n_k);
                if (qe < qa || ke < ka || qa != raw.x || qe != raw.y || ka != raw.z || ke != raw.w) raise_error(p.err, DEV_ERANGE);
            }
            if (!go((uint32_t)max(qe - qa, 0))) break;
            auto tiles = [&](int a, int e, int k0, int k1, int64_t from, int64_t by) {
                PromptTile w;
                w.q0 = a;
                w.k0 = k0;
                w.lk = max(k1 - k0, 0);
                w.shift = w.lk - (e - a);
                for (int64_t r = from * p.tile_tokens; r < e - a; r += by * p.tile_tokens) {
                    w.row0 = (int)r;
                    w.rows = min(p.tile_tokens, e - a - w.row0);
                    const int c = tile_cost(w, p.window) >> p.list_shift;
                    f(w, LIST_BINS - 1 - min(c, LIST_BINS - 1));   // longest in the first bin
                }
            };
            const bool alone = qe - qa <= 4 * p.tile_tokens;
            if (alone) tiles(qa, qe, ka, ke, 0, 1);
            for (uint32_t rest = __ballot_sync(0xffffffffu, !alone); rest; rest &= rest - 1) {
                const int src = __ffs(rest) - 1;
                tiles(__shfl_sync(0xffffffffu, qa, src), __shfl_sync(0xffffffffu, qe, src), __shfl_sync(0xffffffffu, ka, src),
                      __shfl_sync(0xffffffffu, ke, src), lane, 32);
            }
        }
    };
    // Sequences of rising starts have n_q rows together, and their tiles fit the list.  With starts that fall in between,
    // 2^20 sequences may have all rows each: more tiles than the list, 32 bits or one CTA's time hold.  A warp stops when it
    // alone passes n_q, and no tile is worked on.
    auto warp_sum = [](uint32_t n) {
        return ((uint64_t)__reduce_add_sync(0xffffffffu, n >> 16) << 16) + __reduce_add_sync(0xffffffffu, n & 0xffffu);
    };
    uint64_t rows = 0;
    each(
        [&](uint32_t n) {
            rows += warp_sum(n);
            return rows <= p.n_q;
        },
        [&](const PromptTile &, int b) { atomicAdd(&bin[b], 1); });
    if (lane == 0) wrows[warp] = (uint32_t)min(rows, (uint64_t)0xffffffffu);
    __syncthreads();
    if (warp_sum(wrows[lane]) > p.n_q) {
        if (tid == 0) {
            *reinterpret_cast<int *>(p.list) = 0;
            raise_error(p.err, DEV_ERANGE);
        }
        return;
    }
    int sum = bin[tid];
    const int mine = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) wsum[warp] = sum;
    __syncthreads();
    int before = 0;
    for (int k = 0; k < warp; ++k) before += wsum[k];
    bin[tid] = before + sum - mine;
    if (tid == LIST_THREADS - 1) *reinterpret_cast<int *>(p.list) = before + sum;
    __syncthreads();
    each([](uint32_t) { return true; }, [&](const PromptTile &w, int b) {
        list[atomicAdd(&bin[b], 1)] = w;
    });
}

template <bool BF16>
__global__ void __launch_bounds__(Pt::THREADS, 1)
    k_attn_prompt_tc(const AttnPromptParams p, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    using C = Pt;
    constexpr int D = C::D;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int sh[C::THREADS / 32 + 5];
    __shared__ uint32_t tmem_slot;
    // dirty[k & 7] == k + 1: item k of this CTA had values removed; more: a later item's mark lies over item k's, whose
    // rows are then looked through in any case (the guard passes items without a key, and the other query tile's, unhindered)
    __shared__ volatile int abort_flag, dirty[8];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *qs = smem, *ring = smem + 2 * C::TILE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + C::NST * C::STAGE);
    uint64_t *qfull = bars, *qempty = bars + 1, *full = bars + 2, *empty = full + C::NST, *ready = empty + C::NST;
    uint64_t *sfull = ready + C::NST, *pfull = sfull + 2, *ofull = pfull + 2, *done = ofull + 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        for (int i = 0; i < C::NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&ready[i], 2);          // both guard warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 4);          // the tile's four warps
            mbar_init(&ofull[i], 1);
        }
        mbar_init(done, 1);
        abort_flag = 0;
        for (int i = 0; i < 8; ++i) dirty[i] = 0;
        fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmQ)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmK)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmV)) : "memory");
    }
    grid_dep_wait();   // before TMEM is taken: a predecessor that still needs it is waited for
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const uint32_t per_tile = p.n_heads / p.pack;   // items of a tile: groups of packed heads
    __shared__ PromptTile w_one;
    bool one = false;
    if (!p.list) {
        PromptTile w;
        one = prompt_tile<C::THREADS>(p, p.tile_tokens, blockIdx.x / per_tile, blockIdx.x == 0, w, sh);
        if (one && tid == 0) w_one = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint64_t lim = wait_limit(p.wait_ns);
    const uint32_t group = p.n_heads / p.n_kv;
    // items of this CTA: its own, or its share of the list's, the groups of heads of a tile side by side
    const uint32_t n_items = p.list ? (uint32_t)min((uint64_t)*reinterpret_cast<const uint32_t *>(p.list) * per_tile, (uint64_t)0xffff0000u)
                                    : (one ? blockIdx.x + 1 : 0);
    // Every second round of the list is dealt out backwards: the longest of one round goes with the shortest of
    // the next (4096 tokens, 32 heads of 128 on 8: 122 -> 101 us).
    auto item_of = [&](uint32_t round) {
        if (!p.list) return round ? 0xffffffffu : (uint32_t)blockIdx.x;
        return round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : (uint32_t)blockIdx.x);
    };
    auto load_item = [&](uint32_t id) {
        return p.list ? p.list[1 + id / per_tile] : w_one;
    };
    // key tiles [t0[i], t1[i]) that query tile i sees, and [n0, n1) that either sees
    struct Range {
        int t0[2], t1[2], n0, n1;
    };
    auto ranges = [&](const PromptTile &w) {
        Range r;
        r.n0 = INT32_MAX;
        r.n1 = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int ra = p.half * i, rb = min(w.rows, ra + p.half) - 1;
            r.t0[i] = r.t1[i] = 0;
            if (rb >= ra && w.last(rb) >= 0) {
                r.t0[i] = w.first(ra, p.window) / C::BN;
                r.t1[i] = w.last(rb) / C::BN + 1;
                r.n0 = min(r.n0, r.t0[i]);
                r.n1 = max(r.n1, r.t1[i]);
            }
        }
        if (r.n1 == 0) r.n0 = 0;
        return r;
    };

    {
        if (warp == 8) {
            // ------------------------------------------------ TMA producer
            uint32_t fills[C::NST] = {}, q_loads = 0, u = 0;
            auto go = [&](uint64_t *bar, uint32_t parity) {
                return __shfl_sync(0xffffffffu, (int)(!p.withhold && tile_wait(bar, parity, p.err, &abort_flag, lim) && !abort_flag),
                                   0) != 0;
            };
            for (uint32_t round = 0, id; (id = item_of(round)) < n_items; ++round) {
                const PromptTile w = load_item(id);
                const Range r = ranges(w);
                const int head0 = (int)(id % per_tile) * p.pack, kx = head0 / (int)group * D;
                if (r.n1 == r.n0) continue;
                if (go(qempty, (q_loads & 1) ^ 1)) {
                    if (lane == 0) {
                        const int n = w.rows > p.half ? 2 : 1;
                        mbar_arrive_expect_tx(qfull, (uint32_t)(n * C::CH * p.half * p.pack * 128));
                        for (int i = 0; i < n; ++i)
                            for (int c = 0; c < C::CH; ++c)
                                tma_load_3d(qs + i * C::TILE + c * 16384, &tmQ, 64 * c, head0, w.q0 + w.row0 + p.half * i, qfull);
                    }
                    ++q_loads;
                }
                __syncwarp();
                for (int n = r.n0; n <= r.n1; ++n, ++u) {
                    const int st = u % C::NST;
                    if (go(&empty[st], ((u / C::NST) & 1) ^ 1)) {
                        if (lane == 0) {
                            const bool vals = n > r.n0, keys = n < r.n1;
                            mbar_arrive_expect_tx(&full[st], (vals && keys ? 2 : 1) * C::TILE);
                            uint8_t *t = ring + st * C::STAGE;
                            const int y = w.k0 + n * C::BN;
                            for (int c = 0; c < C::CH; ++c) {
                                if (vals) tma_load_2d(t + c * 16384, &tmV, kx + 64 * c, y - C::BN, &full[st]);
                                if (keys) tma_load_2d(t + C::TILE + c * 16384, &tmK, kx + 64 * c, y, &full[st]);
                            }
                        }
                        ++fills[st];
                    }
                    __syncwarp();
                }
            }
            if (abort_flag && lane == 0) {
                // let every copy this warp issued land before the CTA exits
                const uint64_t t_end = global_timer_ns() + WAIT_LIMIT_NS;
                if (q_loads) mbar_drain(qfull, (q_loads - 1u) & 1u, t_end);
                for (int s = 0; s < C::NST; ++s)
                    if (fills[s]) mbar_drain(&full[s], (fills[s] - 1u) & 1u, t_end);
            }
            __syncwarp();
        } else if (warp == 9) {
            // ------------------------------------------------ UMMA issuer
            constexpr uint32_t idS = tc_idesc(128, C::BN, BF16, false), idO = tc_idesc(128, D, BF16, true);
            // addresses in the descriptors count 16 bytes
            const uint64_t dq = sw128_desc(smem_addr(qs)), dk = sw128_desc(smem_addr(ring) + C::TILE),
                           dv = sw128_desc_mn(smem_addr(ring), 16384);
            bool ok = true;
            uint32_t u = 0, q_loads = 0, p_done[2] = {0, 0};
            for (uint32_t round = 0, id; (id = item_of(round)) < n_items; ++round) {
                const PromptTile w = load_item(id);
                const Range r = ranges(w);
                if (r.n1 == r.n0) continue;
                ok = tile_wait(qfull, q_loads & 1, p.err, &abort_flag, lim) && ok;
                ++q_loads;
                for (int n = r.n0; n <= r.n1; ++n, ++u) {    // P V of key tile n - 1, then S of key tile n
                    const int st = u % C::NST;
                    const uint64_t bv = dv + (uint32_t)st * (C::STAGE / 16), bk = dk + (uint32_t)st * (C::STAGE / 16);
                    ok = tile_wait(&ready[st], (u / C::NST) & 1, p.err, &abort_flag, lim) && ok;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const bool pv = n > r.t0[i] && n <= r.t1[i], sc = n >= r.t0[i] && n < r.t1[i];
                        if (pv) {
                            ok = tile_wait(&pfull[i], p_done[i] & 1, p.err, &abort_flag, lim) && ok;
                            ++p_done[i];
                        }
                        tc_fence_after();
                        if (elect_one()) {
                            if (pv && ok) {
#pragma unroll
                                for (int k = 0; k < C::BN / 16; ++k)
                                    tc_mma_f16_ta(tmem + 256 + i * 128, tmem + i * 128 + 8 * k, bv + k * (2048 / 16), idO,
                                                  n - 1 > r.t0[i] || k > 0);
                            }
                            if (sc) {
                                if (ok) {
#pragma unroll
                                    for (int k = 0; k < D / 16; ++k) {
                                        const uint32_t off = ((k / 4) * 16384 + (k % 4) * 32) / 16;
                                        tc_mma_f16(tmem + i * 128, dq + i * (C::TILE / 16) + off, bk + off, idS, k > 0);
                                    }
                                }
                                tc_commit(&sfull[i]);
                            } else if (pv) {
                                tc_commit(&ofull[i]);
                            }
                            if (i == 1 && ok) {
                                tc_commit(&empty[st]);
                                if (n == r.n1 - 1) tc_commit(qempty);
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            if (elect_one()) tc_commit(done);
            __syncwarp();
            tile_wait(done, 0, p.err, nullptr);   // the fixed 2 s limit: TMEM is freed after this
        } else if (warp >= 10) {
            // ------------------------------------------------ V guard
            const int gt = tid - 320;
            uint32_t u = 0;
            int item = 0;
            for (uint32_t round = 0, id; (id = item_of(round)) < n_items; ++round, ++item) {
                const PromptTile w = load_item(id);
                const Range r = ranges(w);
                if (r.n1 == r.n0) continue;
                for (int n = r.n0; n <= r.n1; ++n, ++u) {
                    const int st = u % C::NST;
                    const bool ok = tile_wait(&full[st], (u / C::NST) & 1, p.err, &abort_flag, lim);
                    if (ok && n > r.n0 && w.masked((n - 1) * C::BN, C::BN, p.window)) {
                        prompt_scrub_tile<BF16, C::TILE>(ring + st * C::STAGE, gt, &dirty[item & 7], item + 1);
                        fence_async_smem();
                    }
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(&ready[st]);
                }
            }
        } else {
            // ------------------------------------------------ softmax of tile i, one row a thread
            const int i = warp >> 2, r0 = (warp & 3) * 32;
            const RowOf me(p, i, r0 + lane);
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t tS = tmem + lanes + i * 128, tO = tmem + lanes + 256 + i * 128;
            uint32_t s_seen = 0, o_seen = 0;
            int item = 0;
            for (uint32_t round = 0, id; (id = item_of(round)) < n_items; ++round, ++item) {
                int last, first, w_last, w_first, ta, tb;
                {
                    const PromptTile w = load_item(id);
                    const Range r = ranges(w);
                    last = w.last(me.token);
                    first = w.first(me.token, p.window);
                    // tiles that every row of the warp sees whole need no mask
                    w_last = w.last(RowOf(p, i, r0).token);
                    w_first = w.first(RowOf(p, i, r0 + 31).token, p.window);
                    ta = i ? r.t0[1] : r.t0[0];
                    tb = i ? r.t1[1] : r.t1[0];
                }
                float m = -INFINITY, l = 0.0f;
                for (int n = ta; n < tb; ++n) {
                    tile_wait(&sfull[i], s_seen & 1, p.err, &abort_flag, lim);
                    ++s_seen;
                    tc_fence_after();
                    uint32_t v[128];
                    tc_ld32(tS, v);
                    tc_ld32(tS + 32, v + 32);
                    tc_ld32(tS + 64, v + 64);
                    tc_ld32(tS + 96, v + 96);
                    tc_wait_ld();
                    tc_regs_ready(v);
                    if (n * C::BN + C::BN - 1 > w_last || n * C::BN < w_first) row_mask(v, first - n * C::BN, last - n * C::BN);
                    const float mx = row_max(v) * p.scale_log2;
                    // a first maximum needs no rescaling: O is still zero in that row
                    const bool grow = mx > m + 8.0f;
                    float f = 1.0f;
                    if (grow) {
                        f = m == -INFINITY ? 1.0f : ex2(weight_ref<LAZY_UP<BF16>>(m) - weight_ref<LAZY_UP<BF16>>(mx));
                        m = mx;
                        l *= f;
                    }
                    if (__any_sync(0xffffffffu, f != 1.0f) && n > ta) row_rescale<D>(tO, f);
                    l += row_weights<BF16>(v, p.scale_log2, weight_ref<LAZY_UP<BF16>>(m), tS);
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pfull[i]);
                }
                // ---- results; what does not need O comes before the wait for it
                const PromptTile w = load_item(id);
                const uint32_t head = id % per_tile * p.pack + me.head, kvh = head / group;
                float lse;
                const float f = softmax_finish(weight_ref<LAZY_UP<BF16>>(m), l, p.sinks != nullptr, p.sinks ? p.sinks[head] * 1.4426950408889634f : 0.0f, lse);
                const bool mine = me.used && me.token < w.rows;
                const uint64_t orow = (uint64_t)(w.q0 + w.row0 + me.token) * p.n_heads + head;
                const uint16_t *vp = static_cast<const uint16_t *>(p.v) + (uint64_t)w.k0 * p.v_stride + (uint64_t)kvh * D;
                if (p.lse && mine) p.lse[orow] = lse;
                if (tb > ta) {
                    tile_wait(&ofull[i], o_seen & 1, p.err, &abort_flag, lim);
                    ++o_seen;
                }
                tc_fence_after();
                row_output<D, BF16>(p, w, tO, f, mine, orow, 0, dirty[item & 7] > item ? vp : nullptr, me.token);
                tc_fence_before();   // O is read: the next tile's first P V follows this warp's next arrival
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <bool BF16> cudaError_t launch_tc(const AttnPromptParams &p, int num_sms, cudaStream_t st) {
    static SmemAllowed allowed;
    const cudaError_t es = allow_smem(allowed, reinterpret_cast<const void *>(k_attn_prompt_tc<BF16>), Pt::SMEM);
    if (es != cudaSuccess) return es;
    alignas(64) CUtensorMap tmQ, tmK, tmV;
    if (!encode_3d16_tmap(&tmQ, p.q, Pt::D, p.n_heads, p.n_q, Pt::D, p.q_stride, (uint32_t)p.pack, (uint32_t)p.half, BF16) ||
        (p.n_k && (!encode_rows16_tmap(&tmK, p.k, (uint64_t)p.n_kv * Pt::D, p.n_k, p.k_stride, 128, BF16) ||
                   !encode_rows16_tmap(&tmV, p.v, (uint64_t)p.n_kv * Pt::D, p.n_k, p.v_stride, 128, BF16))))
        return cudaErrorInvalidValue;
    if (!p.n_k) tmK = tmV = tmQ;   // no key tile is loaded
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.list ? (unsigned)num_sms : (unsigned)(p.n_heads / p.pack * (p.n_q / p.tile_tokens + p.n_seq)));
    cfg.blockDim = dim3(Pt::THREADS);
    cfg.dynamicSmemBytes = Pt::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_attn_prompt_tc<BF16>, p, tmQ, tmK, tmV);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

void attn_prompt_tiling(AttnPromptParams &p, int num_sms) {
    p.pack = attn_prompt_pack(p.n_heads / p.n_kv, p.n_kv, p.dim, p.n_q, p.n_seq, num_sms);
    p.half = 128 / p.pack;
    p.tile_tokens = p.half * attn_prompt_halves(p.dim);
}

size_t attn_prompt_list_bytes(const AttnPromptParams &p, int num_sms) {
    const uint64_t tiles = p.n_q / p.tile_tokens + p.n_seq;
    return tiles * (p.n_heads / p.pack) * attn_prompt_parts(p.dim) > (uint64_t)num_sms ? (tiles + 1) * sizeof(PromptTile) : 0;
}

cudaError_t launch_attn_prompt(AttnPromptParams p, void *list, int num_sms, cudaStream_t st) {
    if (list) {
        p.list = static_cast<PromptTile *>(list);
        p.list_cap = p.n_q / p.tile_tokens + p.n_seq;
        for (p.list_shift = 0; (p.n_k / 128 >> p.list_shift) >= LIST_BINS - 1; ++p.list_shift) {}
        const cudaError_t e = launch_dependent(k_attn_prompt_list, p, dim3(1), LIST_THREADS, 0, st);
        if (e != cudaSuccess) return e;
    }
    if (p.dim > 128) return launch_attn_prompt_wide(p, num_sms, st);
    if (p.dim == 64) return launch_attn_prompt_64(p, num_sms, st);
    const bool bf = p.type == Q8_TYPE_BF16;
    return bf ? launch_tc<true>(p, num_sms, st) : launch_tc<false>(p, num_sms, st);
}

}  // namespace q8
