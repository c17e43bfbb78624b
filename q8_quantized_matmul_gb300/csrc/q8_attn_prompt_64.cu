// q8_attn_prompt_64.cu -- attention over whole packed prompts on the 5th-generation tensor cores, heads of 64
// values.
//
// The tiles, roles, list, lazy rescaling and V guard of q8_attn_prompt_tc.cu; what differs is what bounds it.  At 64
// values a key tile's products take the tensor pipe 1050 cycles for both query tiles and the exponentials alone the
// special-function pipes 1024, while the chain S -> softmax -> P V -> next S of one tile took 2500 with one S buffer
// a tile.  O of both tiles takes only 128 TMEM columns here, so there are three S buffers.  The pairs x = 2 (key tile)
// + (query tile) of an item form one sequence; pair x works in buffer x % 3, and S of pair x + 3 is issued right behind
// P V of pair x, in one group: the next scores of a tile are ready when its softmax of the last ones ends.
// Measured: one prompt of 8192 tokens, 32 heads on 8, 250 to 257 us (1.10 PFLOP/s; 2050 cycles a key tile; 274 us with one
// buffer a tile); 12 packed prompts with a window of 1024 85 us (with one buffer 6 more).  Of the 2050 the softmax takes 1350 (probe: a
// warp's step 881 cycles alone, two on a scheduler 1346); the rest is waits for S behind the other tile's group.
// Registers are split 104 / 200 between the roles: with 168 a thread the softmax spills (a step 1150 instead of 885).
// Two issuing warps, one a query tile, gained 1 % on the long prompt and lost 10 % on the short ones.
//
// Barriers by parity.  A wait passes rightly only if the phase before is complete and the one after is not.  S, P and
// P V have two barriers a query tile, its step c (pairs that it takes part in) on c % 2: S of c + 2 follows P V of c,
// so it needs this tile's P of c, as P V of c + 2 needs its P; S of c was waited for before S of c + 2 is, P V of
// c - 2 was committed ahead of S of c, and the issuer waits for every P in order.
#include "q8_attn_prompt_tc.cuh"
#include "q8_kv.h"
#include "q8_launch.h"

namespace q8 {

bool encode_rows16_tmap(CUtensorMap *map, const void *base, uint64_t cols, uint64_t rows, uint64_t row_stride,
                        uint32_t box_rows, bool bf16);
bool encode_3d16_tmap(CUtensorMap *map, const void *base, uint64_t cols, uint64_t n1, uint64_t n2, uint64_t stride1,
                      uint64_t stride2, uint32_t box1, uint32_t box2, bool bf16);

namespace {

struct P64 {
    static constexpr int D = 64, BN = 128;
    static constexpr int TILE = 128 * D * 2;                 // 128 rows of q, k or v: 16 KB
    static constexpr int STAGE = 2 * TILE;                   // the values of key tile u - 2, the keys of key tile u
    static constexpr int NST = 6;
    static constexpr int THREADS = 384;
    static constexpr int NBAR = 2 + 3 * NST + 3 * 4 + 1;
    static constexpr int SMEM = 1024 + 2 * TILE + NST * STAGE + NBAR * 8 + 128;
};

template <bool BF16>
__global__ void __launch_bounds__(P64::THREADS, 1)
    k_attn_prompt_64(const AttnPromptParams p, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    using C = P64;
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
    uint64_t *sfull = ready + C::NST, *odone = sfull + 4, *pfull = odone + 4, *done = pfull + 4;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        for (int i = 0; i < C::NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&ready[i], 2);          // both guard warps
        }
        for (int i = 0; i < 4; ++i) {         // [2 * query tile + step % 2]
            mbar_init(&sfull[i], 1);
            mbar_init(&odone[i], 1);
            mbar_init(&pfull[i], 4);          // the tile's four warps
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
    // the next (4096 tokens, 32 heads of 64 on 8: 93 -> 76 us).
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
        // Units of the ring, an item's N key tiles: unit u = 0 .. N + 1 holds the values u - 2 and the keys u, as far as
        // there are these.
        // registers: 384 threads x 168 of the launch = 128 x 104 + 256 x 200
        if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;\n" ::: "memory");
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
                const int head0 = (int)(id % per_tile) * p.pack, kx = head0 / (int)group * C::D;
                if (r.n1 == r.n0) continue;
                if (go(qempty, (q_loads & 1) ^ 1)) {
                    if (lane == 0) {
                        const int n = w.rows > p.half ? 2 : 1;
                        mbar_arrive_expect_tx(qfull, (uint32_t)(n * p.half * p.pack * 128));
                        for (int i = 0; i < n; ++i)
                            tma_load_3d(qs + i * C::TILE, &tmQ, 0, head0, w.q0 + w.row0 + p.half * i, qfull);
                    }
                    ++q_loads;
                }
                __syncwarp();
                for (int n = r.n0; n < r.n1 + 2; ++n, ++u) {
                    const int st = u % C::NST;
                    if (go(&empty[st], ((u / C::NST) & 1) ^ 1)) {
                        if (lane == 0) {
                            const bool k = n < r.n1, v = n >= r.n0 + 2;
                            uint8_t *dst = ring + st * C::STAGE;
                            if (k || v) mbar_arrive_expect_tx(&full[st], (uint32_t)(k + v) * C::TILE);
                            else mbar_arrive(&full[st]);
                            if (v) tma_load_2d(dst, &tmV, kx, w.k0 + (n - 2) * C::BN, &full[st]);
                            if (k) tma_load_2d(dst + C::TILE, &tmK, kx, w.k0 + n * C::BN, &full[st]);
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
            constexpr uint32_t idS = tc_idesc(128, C::BN, BF16, false), idO = tc_idesc(128, C::D, BF16, true);
            // addresses in the descriptors count 16 bytes
            const uint64_t dq = sw128_desc(smem_addr(qs)), dk = sw128_desc(smem_addr(ring) + C::TILE),
                           dv = sw128_desc_mn(smem_addr(ring), C::TILE);
            bool ok = true;
            uint32_t ub = 0, q_loads = 0;                     // units before the item
            uint32_t cs[2] = {}, cp[2] = {};                  // steps of each query tile whose S, whose P V was issued
            for (uint32_t round = 0, id; (id = item_of(round)) < n_items; ++round) {
                const PromptTile w = load_item(id);
                const Range r = ranges(w);
                const int N = r.n1 - r.n0;
                if (N == 0) continue;
                ok = tile_wait(qfull, q_loads & 1, p.err, &abort_flag, lim) && ok;
                ++q_loads;
                auto ready_unit = [&](uint32_t u) {
                    ok = tile_wait(&ready[u % C::NST], (u / C::NST) & 1, p.err, &abort_flag, lim) && ok;
                };
                auto active = [&](int i, int m) { return m + r.n0 >= r.t0[i] && m + r.n0 < r.t1[i]; };
                // one thread: S of key tile m and query tile i
                auto scores = [&](int i, int m, uint32_t tS, bool sc) {
                    if (sc) {
                        if (ok) {
                            const uint64_t a = dq + i * (C::TILE / 16), b = dk + (ub + m) % C::NST * (C::STAGE / 16);
#pragma unroll
                            for (int k = 0; k < C::D / 16; ++k) tc_mma_f16(tS, a + k * 2, b + k * 2, idS, k > 0);
                        }
                        tc_commit(&sfull[2 * i + (cs[i] & 1)]);
                    }
                    if (i == 1 && m == N - 1 && ok) tc_commit(qempty);
                };
                ready_unit(ub);
                ready_unit(ub + 1);
                tc_fence_after();
                {
                    const bool a0 = active(0, 0), a1 = active(1, 0), a2 = N > 1 && active(0, 1);
                    if (elect_one()) scores(0, 0, tmem, a0);
                    cs[0] += a0;
                    if (elect_one()) {
                        scores(1, 0, tmem + 128, a1);
                        if (ok) tc_commit(&empty[ub % C::NST]);
                    }
                    cs[1] += a1;
                    if (elect_one()) scores(0, 1, tmem + 256, a2);
                    cs[0] += a2;
                    __syncwarp();
                }
                uint32_t tb = tmem;                           // buffer of pair 2 m
#pragma unroll 1
                for (int m = 0; m < N; ++m) {
                    ready_unit(ub + m + 2);
                    const uint64_t b = dv + (ub + m + 2) % C::NST * (C::STAGE / 16);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // P V of pair 2 m + i; S of the pair three on: the other query tile, key tile m + 1 + i
                        const int ms = m + 1 + i;
                        const bool pv = active(i, m), sc = ms < N && active(1 - i, ms), more = m + r.n0 > r.t0[i];
                        if (pv) ok = tile_wait(&pfull[2 * i + (cp[i] & 1)], (cp[i] >> 1) & 1, p.err, &abort_flag, lim) && ok;
                        tc_fence_after();
                        if (elect_one()) {
                            if (pv) {
                                if (ok) {
#pragma unroll
                                    for (int k = 0; k < C::BN / 16; ++k)
                                        tc_mma_f16_ta(tmem + 384 + i * 64, tb + 8 * k, b + k * (2048 / 16), idO, more || k > 0);
                                }
                                tc_commit(&odone[2 * i + (cp[i] & 1)]);
                            }
                            if (ms < N) scores(1 - i, ms, tb, sc);
                            // the keys m + 1 are through with pair 2 m, the last values with the last pair
                            if (ok && (i == 0 || m == N - 1)) tc_commit(&empty[(ub + m + 1 + i) % C::NST]);
                        }
                        __syncwarp();
                        cp[i] += pv;
                        cs[1 - i] += sc;
                        tb = tb == tmem + 256 ? tmem : tb + 128;
                    }
                }
                ub += N + 2;
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
                for (int n = r.n0; n < r.n1 + 2; ++n, ++u) {
                    const int st = u % C::NST;
                    const bool ok = tile_wait(&full[st], (u / C::NST) & 1, p.err, &abort_flag, lim);
                    if (ok && n >= r.n0 + 2 && w.masked((n - 2) * C::BN, C::BN, p.window)) {
                        prompt_scrub_tile<BF16, C::TILE>(ring + st * C::STAGE, gt, &dirty[item & 7], item + 1);
                        fence_async_smem();
                    }
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(&ready[st]);
                }
            }
        } else {
            // ------------------------------------------------ softmax of tile i, one row a thread
            asm volatile("setmaxnreg.inc.sync.aligned.u32 200;\n" ::: "memory");
            const int i = warp >> 2, r0 = (warp & 3) * 32;
            const RowOf me(p, i, r0 + lane);
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t tO = tmem + lanes + 384 + i * 64;
            uint32_t c = 0;                                   // this tile's steps
            int item = 0;
            for (uint32_t round = 0, id; (id = item_of(round)) < n_items; ++round, ++item) {
                int last, first, w_last, w_first, ta, tb;   // [ta, tb): this tile's key tiles
                uint32_t tS;                                  // buffer of the next one
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
                    tS = tmem + lanes + (2 * (ta - r.n0) + i) % 3 * 128;
                }
                float m = -INFINITY, l = 0.0f;
#pragma unroll 1
                for (int n = ta; n < tb; ++n) {
                    tile_wait(&sfull[i * 2 + (c & 1)], (c >> 1) & 1, p.err, &abort_flag, lim);
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
                    float f = 1.0f;
                    if (mx > m + 8.0f) {
                        f = m == -INFINITY ? 1.0f : ex2(weight_ref<LAZY_UP<BF16>>(m) - weight_ref<LAZY_UP<BF16>>(mx));
                        m = mx;
                        l *= f;
                    }
                    if (__any_sync(0xffffffffu, f != 1.0f) && n > ta) {
                        tile_wait(&odone[i * 2 + ((c - 1) & 1)], ((c - 1) >> 1) & 1, p.err, &abort_flag, lim);   // P V of the step before
                        tc_fence_after();
                        row_rescale<C::D>(tO, f);
                    }
                    l += row_weights<BF16>(v, p.scale_log2, weight_ref<LAZY_UP<BF16>>(m), tS);
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pfull[i * 2 + (c & 1)]);
                    ++c;
                    tS = tS >= tmem + lanes + 128 ? tS - 128 : tS + 256;   // two pairs on
                }
                // ---- results; what does not need O comes before the wait for it
                const PromptTile w = load_item(id);
                const uint32_t head = id % per_tile * p.pack + me.head, kvh = head / group;
                float lse;
                const float f = softmax_finish(weight_ref<LAZY_UP<BF16>>(m), l, p.sinks != nullptr, p.sinks ? p.sinks[head] * 1.4426950408889634f : 0.0f, lse);
                const bool mine = me.used && me.token < w.rows;
                const uint64_t orow = (uint64_t)(w.q0 + w.row0 + me.token) * p.n_heads + head;
                const uint16_t *vp = static_cast<const uint16_t *>(p.v) + (uint64_t)w.k0 * p.v_stride + (uint64_t)kvh * C::D;
                if (p.lse && mine) p.lse[orow] = lse;
                if (tb > ta) tile_wait(&odone[i * 2 + ((c - 1) & 1)], ((c - 1) >> 1) & 1, p.err, &abort_flag, lim);
                tc_fence_after();
                row_output<C::D, BF16>(p, w, tO, f, mine, orow, 0, dirty[item & 7] > item ? vp : nullptr, me.token);
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

template <bool BF16> cudaError_t launch_64(const AttnPromptParams &p, int num_sms, cudaStream_t st) {
    static SmemAllowed allowed;
    const cudaError_t es = allow_smem(allowed, reinterpret_cast<const void *>(k_attn_prompt_64<BF16>), P64::SMEM);
    if (es != cudaSuccess) return es;
    alignas(64) CUtensorMap tmQ, tmK, tmV;
    if (!encode_3d16_tmap(&tmQ, p.q, P64::D, p.n_heads, p.n_q, P64::D, p.q_stride, (uint32_t)p.pack, (uint32_t)p.half, BF16) ||
        (p.n_k && (!encode_rows16_tmap(&tmK, p.k, (uint64_t)p.n_kv * P64::D, p.n_k, p.k_stride, 128, BF16) ||
                   !encode_rows16_tmap(&tmV, p.v, (uint64_t)p.n_kv * P64::D, p.n_k, p.v_stride, 128, BF16))))
        return cudaErrorInvalidValue;
    if (!p.n_k) tmK = tmV = tmQ;   // no key tile is loaded
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.list ? (unsigned)num_sms : (unsigned)(p.n_heads / p.pack * (p.n_q / p.tile_tokens + p.n_seq)));
    cfg.blockDim = dim3(P64::THREADS);
    cfg.dynamicSmemBytes = P64::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_attn_prompt_64<BF16>, p, tmQ, tmK, tmV);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_attn_prompt_64(const AttnPromptParams &p, int num_sms, cudaStream_t st) {
    return p.type == Q8_TYPE_BF16 ? launch_64<true>(p, num_sms, st) : launch_64<false>(p, num_sms, st);
}

}  // namespace q8
