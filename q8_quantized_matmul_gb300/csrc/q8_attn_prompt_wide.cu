// q8_attn_prompt_wide.cu -- attention over whole packed prompts on the 5th-generation tensor cores, heads of
// 256 or 512 values.
//
// A work item is 128 rows (queries of one head, or of several packed heads) and 256 of their output dims (heads of 512: two items, which both
// compute the scores).  TMEM: two buffers of S (128 columns each) and O (256).  S of key tile n + 1 is issued
// before P V of tile n, so the softmax of a tile (about 1000 cycles) runs under the next one's S (2048 cycles at
// 512 values, 1024 at 256) and the tensor pipe does not wait for it.  Operands stream through a ring of slots of
// 128 keys x 128 dims (32 KB); at 512 values q takes 128 KB of shared memory and three slots are left.  Reading
// both operands of S there (128 bytes a cycle) and filling the ring bound the kernel: at 512 values a key tile
// moves 512 KB through shared memory, 4096 cycles, for three quarters as many of products.  One prompt of 4096
// tokens with 16 heads of 256 on one takes 105 us (1.31 PFLOP/s), of 2048 with 64 heads of 512 339 us (0.81).
//
// Roles, list of tiles, lazy rescaling and the V guard are those of q8_attn_prompt_tc.cu.  O is rescaled only
// after the P V before has ended (its own barrier, since S of the next tile no longer implies it).
#include "q8_attn_prompt_tc.cuh"
#include "q8_kv.h"
#include "q8_launch.h"

namespace q8 {

bool encode_rows16_tmap(CUtensorMap *map, const void *base, uint64_t cols, uint64_t rows, uint64_t row_stride,
                        uint32_t box_rows, bool bf16);
bool encode_3d16_tmap(CUtensorMap *map, const void *base, uint64_t cols, uint64_t n1, uint64_t n2, uint64_t stride1,
                      uint64_t stride2, uint32_t box1, uint32_t box2, bool bf16);

namespace {

template <int D> struct Pw {
    static constexpr int BN = 128, BM = 128, DV = 256, PARTS = D / DV;
    static constexpr int CHUNK = 128 * 128, SLOT = 2 * CHUNK;   // 128 rows x 64 dims; two of them
    static constexpr int KS = D / 128, VS = DV / 128;        // slots of a key tile, of a value tile
    static constexpr int QBYTES = BM * D * 2;
    static constexpr int NST = D == 512 ? 3 : 4;
    static constexpr int THREADS = 256;
    static constexpr int NBAR = 2 + 3 * NST + 2 + 2 + 2 + 1;
    static constexpr int SMEM = 1024 + QBYTES + NST * SLOT + NBAR * 8 + 64;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int D, bool BF16>
__global__ void __launch_bounds__(Pw<D>::THREADS, 1)
    k_attn_prompt_wide(const AttnPromptParams p, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    using C = Pw<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int sh[C::THREADS / 32 + 5];
    __shared__ uint32_t tmem_slot;
    // dirty[k & 7] == k + 1: item k of this CTA had values removed; more: a later item's mark lies over item k's, whose
    // rows are then looked through in any case (the guard passes items without a key, and the other query tile's, unhindered)
    __shared__ volatile int abort_flag, dirty[8];
    __shared__ PromptTile w_one;
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *qs = smem, *ring = smem + C::QBYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + C::NST * C::SLOT);
    uint64_t *qfull = bars, *qempty = bars + 1, *full = bars + 2, *empty = full + C::NST, *ready = empty + C::NST;
    uint64_t *sfull = ready + C::NST, *pfull = sfull + 2, *odone = pfull + 2, *done = odone + 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        for (int i = 0; i < C::NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&ready[i], 2);          // both guard warps
        }
        for (int i = 0; i < 2; ++i) {         // by key tile: the softmax may be one ahead of P V
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 4);
            mbar_init(&odone[i], 1);
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
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const uint32_t per_tile = p.n_heads / p.pack * C::PARTS;   // items of a tile: groups of packed heads, their parts side by side
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
    const uint32_t n_items = p.list ? (uint32_t)min((uint64_t)*reinterpret_cast<const uint32_t *>(p.list) * per_tile, (uint64_t)0xffff0000u)
                                    : (one ? blockIdx.x + 1 : 0);
    // Every second round of the list is dealt out backwards: the longest of one round goes with the shortest of
    // the next (4096 tokens, 16 heads of 256 on one: 126 -> 106 us).
    auto item_of = [&](uint32_t round) {
        if (!p.list) return round ? 0xffffffffu : (uint32_t)blockIdx.x;
        return round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : (uint32_t)blockIdx.x);
    };
    auto load_item = [&](uint32_t id) { return p.list ? p.list[1 + id / per_tile] : w_one; };
    // key tiles [n0, n1) that the rows see
    auto range = [&](const PromptTile &w, int &n0, int &n1) {
        n0 = n1 = 0;
        if (w.last(w.rows - 1) >= 0) {
            n0 = w.first(0, p.window) / C::BN;
            n1 = w.last(w.rows - 1) / C::BN + 1;
        }
    };
    // slots in the order of their use: keys of n0, then for each n the keys of n + 1 and the values of n

    if (warp == 4) {
        // ------------------------------------------------ TMA producer
        uint32_t fills[C::NST] = {}, q_loads = 0, u = 0;
        auto go = [&](uint64_t *bar, uint32_t parity) {
            return __shfl_sync(0xffffffffu, (int)(!p.withhold && tile_wait(bar, parity, p.err, &abort_flag, lim) && !abort_flag), 0) != 0;
        };
        auto slots = [&](const CUtensorMap *map, int n_slots, int x, int y) {
            for (int j = 0; j < n_slots; ++j, ++u) {
                const int st = u % C::NST;
                if (go(&empty[st], ((u / C::NST) & 1) ^ 1)) {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&full[st], C::SLOT);
                        for (int c = 0; c < 2; ++c)
                            tma_load_2d(ring + st * C::SLOT + c * C::CHUNK, map, x + j * 128 + c * 64, y, &full[st]);
                    }
                    ++fills[st];
                }
                __syncwarp();
            }
        };
        for (uint32_t round = 0, id; (id = item_of(round)) < n_items; ++round) {
            const PromptTile w = load_item(id);
            int n0, n1;
            range(w, n0, n1);
            if (n1 == n0) continue;
            const uint32_t r = id % per_tile, head0 = r / C::PARTS * p.pack;
            const int kx = (int)(head0 / group) * D, vx = kx + (int)(r % C::PARTS) * C::DV;
            if (go(qempty, (q_loads & 1) ^ 1)) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(qfull, (uint32_t)(D / 64 * p.half * p.pack * 128));
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(qs + c * C::CHUNK, &tmQ, 64 * c, (int)head0, w.q0 + w.row0, qfull);
                }
                ++q_loads;
            }
            __syncwarp();
            slots(&tmK, C::KS, kx, w.k0 + n0 * C::BN);
            for (int n = n0; n < n1; ++n) {
                if (n + 1 < n1) slots(&tmK, C::KS, kx, w.k0 + (n + 1) * C::BN);
                slots(&tmV, C::VS, vx, w.k0 + n * C::BN);
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
    } else if (warp == 5) {
        // ------------------------------------------------ UMMA issuer
        constexpr uint32_t idS = tc_idesc(128, C::BN, BF16), idO = tc_idesc(128, 128, BF16, true);
        // addresses in the descriptors count 16 bytes
        const uint64_t dq = sw128_desc(smem_addr(qs)), dk = sw128_desc(smem_addr(ring)),
                       dv = sw128_desc_mn(smem_addr(ring), C::CHUNK);
        bool ok = true;
        uint32_t u = 0, q_loads = 0, nt = 0;   // nt: key tiles so far, over all items
        auto scores = [&](uint32_t t, bool last) {
            const uint32_t tS = tmem + (t & 1) * 128;
            for (int j = 0; j < C::KS; ++j, ++u) {
                const int st = u % C::NST;
                ok = tile_wait(&ready[st], (u / C::NST) & 1, p.err, &abort_flag, lim) && ok;
                tc_fence_after();
                if (elect_one()) {
                    if (ok) {
                        const uint64_t a = dq + (uint32_t)j * (C::SLOT / 16), b = dk + (uint32_t)st * (C::SLOT / 16);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t off = ((k / 4) * C::CHUNK + (k % 4) * 32) / 16;
                            tc_mma_f16(tS, a + off, b + off, idS, j > 0 || k > 0);
                        }
                        tc_commit(&empty[st]);
                    }
                    if (j == C::KS - 1) {
                        tc_commit(&sfull[t & 1]);
                        if (last && ok) tc_commit(qempty);
                    }
                }
                __syncwarp();
            }
        };
        for (uint32_t round = 0, id; (id = item_of(round)) < n_items; ++round) {
            const PromptTile w = load_item(id);
            int n0, n1;
            range(w, n0, n1);
            if (n1 == n0) continue;
            ok = tile_wait(qfull, q_loads & 1, p.err, &abort_flag, lim) && ok;
            ++q_loads;
            scores(nt, n0 + 1 == n1);
            for (int n = n0; n < n1; ++n, ++nt) {
                if (n + 1 < n1) scores(nt + 1, n + 2 == n1);
                ok = tile_wait(&pfull[nt & 1], (nt >> 1) & 1, p.err, &abort_flag, lim) && ok;
                for (int j = 0; j < C::VS; ++j, ++u) {
                    const int st = u % C::NST;
                    ok = tile_wait(&ready[st], (u / C::NST) & 1, p.err, &abort_flag, lim) && ok;
                    tc_fence_after();
                    if (elect_one()) {
                        if (ok) {
                            const uint64_t b = dv + (uint32_t)st * (C::SLOT / 16);
#pragma unroll
                            for (int k = 0; k < C::BN / 16; ++k)
                                tc_mma_f16_ta(tmem + 256 + j * 128, tmem + (nt & 1) * 128 + 8 * k, b + k * (2048 / 16), idO,
                                              n > n0 || k > 0);
                            tc_commit(&empty[st]);
                        }
                        if (j == C::VS - 1) tc_commit(&odone[nt & 1]);
                    }
                    __syncwarp();
                }
            }
        }
        if (elect_one()) tc_commit(done);
        __syncwarp();
        tile_wait(done, 0, p.err, nullptr);   // the fixed 2 s limit: TMEM is freed after this
    } else if (warp >= 6) {
        // ------------------------------------------------ V guard
        const int gt = tid - 192;
        uint32_t u = 0;
        int item = 0;
        auto pass = [&](int n_slots, bool scrub) {
            for (int j = 0; j < n_slots; ++j, ++u) {
                const int st = u % C::NST;
                const bool ok = tile_wait(&full[st], (u / C::NST) & 1, p.err, &abort_flag, lim);
                if (ok && scrub) {
                    prompt_scrub_tile<BF16, C::SLOT>(ring + st * C::SLOT, gt, &dirty[item & 7], item + 1);
                    fence_async_smem();
                }
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(&ready[st]);
            }
        };
        for (uint32_t round = 0, id; (id = item_of(round)) < n_items; ++round, ++item) {
            const PromptTile w = load_item(id);
            int n0, n1;
            range(w, n0, n1);
            if (n1 == n0) continue;
            pass(C::KS, false);
            for (int n = n0; n < n1; ++n) {
                if (n + 1 < n1) pass(C::KS, false);
                pass(C::VS, w.masked(n * C::BN, C::BN, p.window));
            }
        }
    } else {
        // ------------------------------------------------ softmax, one row a thread
        const RowOf me(p, 0, tid);
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const uint32_t tO = tmem + lanes + 256;
        uint32_t nt = 0;
        int item = 0;
        // P V of key tile t has ended.  The one two before it had when S of tile t was complete, so the parity
        // tells the two apart.
        auto p_v_done = [&](uint32_t t) { tile_wait(&odone[t & 1], (t >> 1) & 1, p.err, &abort_flag, lim); };
        for (uint32_t round = 0, id; (id = item_of(round)) < n_items; ++round, ++item) {
            int last, first, w_last, w_first, n0, n1;
            {
                const PromptTile w = load_item(id);
                range(w, n0, n1);
                last = w.last(me.token);
                first = w.first(me.token, p.window);
                // tiles that every row of the warp sees whole need no mask
                w_last = w.last(RowOf(p, 0, warp * 32).token);
                w_first = w.first(RowOf(p, 0, warp * 32 + 31).token, p.window);
            }
            float m = -INFINITY, l = 0.0f;
            for (int n = n0; n < n1; ++n, ++nt) {
                const uint32_t tS = tmem + lanes + (nt & 1) * 128;
                tile_wait(&sfull[nt & 1], (nt >> 1) & 1, p.err, &abort_flag, lim);
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
                if (__any_sync(0xffffffffu, f != 1.0f) && n > n0) {
                    p_v_done(nt - 1);
                    tc_fence_after();
                    row_rescale<C::DV>(tO, f);
                }
                l += row_weights<BF16>(v, p.scale_log2, weight_ref<LAZY_UP<BF16>>(m), tS);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[nt & 1]);
            }
            // ---- results; what does not need O comes before the wait for it
            const PromptTile w = load_item(id);
            const uint32_t r = id % per_tile, head = r / C::PARTS * p.pack + me.head, kvh = head / group;
            const int d0 = (int)(r % C::PARTS) * C::DV;
            float lse;
            const float f = softmax_finish(weight_ref<LAZY_UP<BF16>>(m), l, p.sinks != nullptr, p.sinks ? p.sinks[head] * 1.4426950408889634f : 0.0f, lse);
            const bool mine = me.used && me.token < w.rows;
            const uint64_t orow = (uint64_t)(w.q0 + w.row0 + me.token) * p.n_heads + head;
            const uint16_t *vp = static_cast<const uint16_t *>(p.v) + (uint64_t)w.k0 * p.v_stride + (uint64_t)kvh * D;
            if (p.lse && mine && d0 == 0) p.lse[orow] = lse;
            if (n1 > n0) p_v_done(nt - 1);
            tc_fence_after();
            row_output<C::DV, BF16>(p, w, tO, f, mine, orow, d0, dirty[item & 7] > item ? vp : nullptr, me.token);
            tc_fence_before();   // O is read: the next item's first P V follows this warp's next arrival
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <int D, bool BF16> cudaError_t launch_wide(const AttnPromptParams &p, int num_sms, cudaStream_t st) {
    static SmemAllowed allowed;
    const cudaError_t es = allow_smem(allowed, reinterpret_cast<const void *>(k_attn_prompt_wide<D, BF16>), Pw<D>::SMEM);
    if (es != cudaSuccess) return es;
    alignas(64) CUtensorMap tmQ, tmK, tmV;
    if (!encode_3d16_tmap(&tmQ, p.q, D, p.n_heads, p.n_q, D, p.q_stride, (uint32_t)p.pack, (uint32_t)p.half, BF16) ||
        (p.n_k && (!encode_rows16_tmap(&tmK, p.k, (uint64_t)p.n_kv * D, p.n_k, p.k_stride, 128, BF16) ||
                   !encode_rows16_tmap(&tmV, p.v, (uint64_t)p.n_kv * D, p.n_k, p.v_stride, 128, BF16))))
        return cudaErrorInvalidValue;
    if (!p.n_k) tmK = tmV = tmQ;   // no key tile is loaded
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.list ? (unsigned)num_sms : (unsigned)(p.n_heads / p.pack * Pw<D>::PARTS * (p.n_q / p.tile_tokens + p.n_seq)));
    cfg.blockDim = dim3(Pw<D>::THREADS);
    cfg.dynamicSmemBytes = Pw<D>::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_attn_prompt_wide<D, BF16>, p, tmQ, tmK, tmV);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_attn_prompt_wide(const AttnPromptParams &p, int num_sms, cudaStream_t st) {
    const bool bf = p.type == Q8_TYPE_BF16;
    if (p.dim == 256) return bf ? launch_wide<256, true>(p, num_sms, st) : launch_wide<256, false>(p, num_sms, st);
    return bf ? launch_wide<512, true>(p, num_sms, st) : launch_wide<512, false>(p, num_sms, st);
}

}  // namespace q8
