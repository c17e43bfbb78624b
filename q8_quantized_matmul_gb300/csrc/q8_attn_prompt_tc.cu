// q8_attn_prompt_tc.cu -- attention over whole packed prompts on the 5th-generation tensor cores,
// heads of 64 or 128 values.
//
// A CTA works on 256 query rows of one head as two tiles of 128 rows, over key tiles of 128.  Per key
// tile and query tile: S = Q K^T (D/16 UMMAs) into 128 TMEM columns; one thread per row reads its S,
// keeps the running maximum m and sum l, writes P = 2^(S - m) as 16-bit pairs over S; O += P V
// (8 UMMAs, P from TMEM) into D further columns.  S of both tiles (256 columns) and O of both (2 D) fill
// the SM's 512 columns.  While the threads of one tile work on its softmax the tensor cores run the
// other tile's products, so the two overlap: at D = 128 a key tile costs the tensor pipe about 2048
// cycles for both query tiles and the softmax warps about half that; at D = 64 they are even.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 since the last time (the weights
// then stay below 2^8, harmless in either 16-bit type); the result is the same sum in other units.  The
// threads of a tile do that themselves: S of the next key tile is complete only after this tile's P V is,
// so O is at rest between the two.
//
// Warps: 0-3 and 4-7 the softmax of the two tiles (thread = row = TMEM lane), 8 the TMA producer, 9 the
// UMMA issuer, 10-11 the V guard.  The guard holds every V tile until it has removed values that are not
// finite from tiles that some rows may not see (0 times infinity would reach them); they are added at the
// end to the rows that do see them (prompt_restore).
//
// Every wait is bounded; after one expires nothing more is issued and copies in flight are drained.
#include "q8_attn.cuh"
#include "q8_attn_prompt.cuh"
#include "q8_kv.h"
#include "q8_tcgen05.cuh"

namespace q8 {

bool encode_rows16_tmap(CUtensorMap *map, const void *base, uint64_t cols, uint64_t rows, uint64_t row_stride,
                        uint32_t box_rows, bool bf16);

namespace {

template <int D> struct Pt {
    static constexpr int BN = 128, BM = 256;
    static constexpr int CH = D / 64;                        // 64-value chunks of a row, 16 KB a chunk of 128 rows
    static constexpr int TILE = 128 * D * 2;
    // stage u holds the values of key tile u - 1 and the keys of tile u, which are used in one go
    static constexpr int STAGE = 2 * TILE;
    static constexpr int NST = D == 128 ? 2 : 4;
    static constexpr int THREADS = 384;
    static constexpr int NBAR = 1 + 3 * NST + 2 + 2 + 2 + 1;
    static constexpr int SMEM = 1024 + 2 * TILE + NST * STAGE + NBAR * 8 + 128;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// 32 fp32 output values of one thread's row, columns d0 ..
__device__ __forceinline__ void store_row32(const AttnPromptParams &p, uint64_t row, int d0, const float *y) {
    const uint64_t i0 = row * p.dim + d0;
    if (p.out_type == Q8_TYPE_Q8_0) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) amax = fmaxf(amax, fabsf(y[i]));
        const float d = __fdiv_rn(amax, 127.0f);
        uint16_t *dst = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(p.out) + i0 / QK * QB);
        dst[0] = d != 0.0f ? __half_as_ushort(__float2half_rn(d)) : 0;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const int a = d != 0.0f ? (int)roundf(__fdiv_rn(y[2 * i], d)) : 0;
            const int b = d != 0.0f ? (int)roundf(__fdiv_rn(y[2 * i + 1], d)) : 0;
            dst[1 + i] = (uint16_t)((a & 0xff) | (b & 0xff) << 8);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = y[8 * i + e];
            store_out8(p.out, p.out_type, i0 + 8 * i, x, true);
        }
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(Pt<D>::THREADS, 1)
    k_attn_prompt_tc(const AttnPromptParams p, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    using C = Pt<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int sh[C::THREADS / 32 + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag, dirty;
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *qs = smem, *ring = smem + 2 * C::TILE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + C::NST * C::STAGE);
    uint64_t *qfull = bars, *full = bars + 1, *empty = full + C::NST, *ready = empty + C::NST;
    uint64_t *sfull = ready + C::NST, *pfull = sfull + 2, *ofull = pfull + 2, *done = ofull + 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        mbar_init(qfull, 1);
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
        dirty = 0;
        fence_mbar_init();
    }
    grid_dep_wait();   // before TMEM is taken: a predecessor that still needs it is waited for
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    PromptTile w;
    const bool any = prompt_tile<C::THREADS>(p, C::BM, blockIdx.y, blockIdx.x + blockIdx.y == 0, w, sh);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint64_t lim = wait_limit(p.wait_ns);
    const uint32_t head = blockIdx.x, kvh = head / (p.n_heads / p.n_kv);

    if (any) {
        // key tiles [t0[i], t1[i]) that query tile i sees, and [n0, n1) that either sees
        int t0[2], t1[2], n0 = INT32_MAX, n1 = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int ra = 128 * i, rb = min(w.rows, ra + 128) - 1;
            t0[i] = t1[i] = 0;
            if (rb >= ra && w.last(rb) >= 0) {
                t0[i] = w.first(ra, p.window) / C::BN;
                t1[i] = w.last(rb) / C::BN + 1;
                n0 = min(n0, t0[i]);
                n1 = max(n1, t1[i]);
            }
        }
        if (n1 == 0) n0 = 0;

        if (warp == 8) {
            // ------------------------------------------------ TMA producer
            uint32_t fills[C::NST] = {};
            bool q_loaded = false;
            if (n1 > n0 && !p.withhold) {
                q_loaded = true;
                if (lane == 0) {
                    const bool two = w.rows > 128;
                    mbar_arrive_expect_tx(qfull, (two ? 2 : 1) * C::TILE);
                    for (int i = 0; i < (two ? 2 : 1); ++i)
                        for (int c = 0; c < C::CH; ++c)
                            tma_load_2d(qs + i * C::TILE + c * 16384, &tmQ, (int)head * D + 64 * c, w.q0 + w.row0 + 128 * i,
                                        qfull);
                }
                __syncwarp();
            }
            for (int u = 0; u <= n1 - n0 && n1 > n0; ++u) {
                const int st = u % C::NST;
                if (__shfl_sync(0xffffffffu, (int)(!p.withhold && mbar_wait(&empty[st], ((u / C::NST) & 1) ^ 1, p.err, &abort_flag, lim) &&
                                                   !abort_flag), 0)) {
                    if (lane == 0) {
                        const bool vals = u > 0, keys = u < n1 - n0;
                        mbar_arrive_expect_tx(&full[st], (vals && keys ? 2 : 1) * C::TILE);
                        uint8_t *t = ring + st * C::STAGE;
                        const int y = w.k0 + (n0 + u) * C::BN;
                        for (int c = 0; c < C::CH; ++c) {
                            if (vals) tma_load_2d(t + c * 16384, &tmV, (int)kvh * D + 64 * c, y - C::BN, &full[st]);
                            if (keys) tma_load_2d(t + C::TILE + c * 16384, &tmK, (int)kvh * D + 64 * c, y, &full[st]);
                        }
                    }
                    ++fills[st];
                }
                __syncwarp();
            }
            if (abort_flag && lane == 0) {
                // let every copy this warp issued land before the CTA exits
                const uint64_t t_end = global_timer_ns() + WAIT_LIMIT_NS;
                if (q_loaded) mbar_drain(qfull, 0, t_end);
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
            bool ok = n1 == n0 || mbar_wait(qfull, 0, p.err, &abort_flag, lim);
            for (int u = 0; u <= n1 - n0 && n1 > n0; ++u) {
                const int st = u % C::NST, n = n0 + u;       // P V of key tile n - 1, then S of key tile n
                const uint64_t bv = dv + (uint32_t)st * (C::STAGE / 16), bk = dk + (uint32_t)st * (C::STAGE / 16);
                ok = mbar_wait(&ready[st], (u / C::NST) & 1, p.err, &abort_flag, lim) && ok;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool pv = n > t0[i] && n <= t1[i], sc = n >= t0[i] && n < t1[i];
                    if (pv) ok = mbar_wait(&pfull[i], (n - 1 - t0[i]) & 1, p.err, &abort_flag, lim) && ok;
                    tc_fence_after();
                    if (elect_one()) {
                        if (pv && ok) {
#pragma unroll
                            for (int k = 0; k < C::BN / 16; ++k)
                                tc_mma_f16_ta(tmem + 256 + i * 128, tmem + i * 128 + 8 * k, bv + k * (2048 / 16), idO,
                                              n - 1 > t0[i] || k > 0);
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
                        if (i == 1 && ok) tc_commit(&empty[st]);
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) tc_commit(done);
            __syncwarp();
            mbar_wait(done, 0, p.err, nullptr);   // the fixed 2 s limit: TMEM is freed after this
        } else if (warp >= 10) {
            // ------------------------------------------------ V guard
            const int gt = tid - 320;
            for (int u = 0; u <= n1 - n0 && n1 > n0; ++u) {
                const int st = u % C::NST;
                const bool ok = mbar_wait(&full[st], (u / C::NST) & 1, p.err, &abort_flag, lim);
                if (ok && u > 0 && w.masked((n0 + u - 1) * C::BN, C::BN, p.window)) {
                    uint4 *t = reinterpret_cast<uint4 *>(ring + st * C::STAGE);
#pragma unroll 4
                    for (int i = gt; i < C::TILE / 16; i += 64) {
                        uint4 x = t[i];
                        if (prompt_scrub<BF16>(x)) {
                            t[i] = x;
                            dirty = 1;
                        }
                    }
                    fence_async_smem();
                }
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(&ready[st]);
            }
        } else {
            // ------------------------------------------------ softmax of tile i, one row a thread
            const int i = warp >> 2, row = i * 128 + (warp & 3) * 32 + lane;
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t tS = tmem + lanes + i * 128, tO = tmem + lanes + 256 + i * 128;
            const int last = w.last(row), first = w.first(row, p.window);
            // tiles that every row of the warp sees whole need no mask
            const int w_last = w.last(i * 128 + (warp & 3) * 32), w_first = w.first(i * 128 + (warp & 3) * 32 + 31, p.window);
            const int ta = i ? t0[1] : t0[0], tb = i ? t1[1] : t1[0];
            float m = -INFINITY, l = 0.0f;
            for (int n = ta; n < tb; ++n) {
                mbar_wait(&sfull[i], (n - ta) & 1, p.err, &abort_flag, lim);
                tc_fence_after();
                uint32_t v[128];
                tc_ld32(tS, v);
                tc_ld32(tS + 32, v + 32);
                tc_ld32(tS + 64, v + 64);
                tc_ld32(tS + 96, v + 96);
                tc_wait_ld();
                tc_regs_ready(v);
                if (n * C::BN + C::BN - 1 > w_last || n * C::BN < w_first) {
                    const int hi = last - n * C::BN, lo = first - n * C::BN;   // columns lo .. hi are seen
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        // bits of the 32 columns from 32 b on
                        const int h = hi + 1 - 32 * b, g = lo - 32 * b;
                        const uint32_t below = h >= 32 ? 0xffffffffu : (h <= 0 ? 0u : (1u << h) - 1u);
                        const uint32_t seen = g <= 0 ? below : (g >= 32 ? 0u : below & (0xffffffffu << g));
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!(seen & (1u << c))) v[32 * b + c] = 0xff800000u;
                    }
                }
                float x0 = __uint_as_float(v[0]), x1 = __uint_as_float(v[1]), x2 = __uint_as_float(v[2]), x3 = __uint_as_float(v[3]);
#pragma unroll
                for (int c = 4; c < 124; c += 8) {
                    x0 = max3(x0, __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
                    x1 = max3(x1, __uint_as_float(v[c + 2]), __uint_as_float(v[c + 3]));
                    x2 = max3(x2, __uint_as_float(v[c + 4]), __uint_as_float(v[c + 5]));
                    x3 = max3(x3, __uint_as_float(v[c + 6]), __uint_as_float(v[c + 7]));
                }
                x0 = max3(x0, __uint_as_float(v[124]), __uint_as_float(v[125]));
                x1 = max3(x1, __uint_as_float(v[126]), __uint_as_float(v[127]));
                const float mx = max3(fmaxf(x0, x1), x2, x3) * p.scale_log2;
                // a first maximum needs no rescaling: O is still zero in that row
                const bool grow = mx > m + 8.0f;
                float f = 1.0f;
                if (grow) {
                    f = m == -INFINITY ? 1.0f : ex2(m - mx);
                    m = mx;
                    l *= f;
                }
                if (__any_sync(0xffffffffu, f != 1.0f) && n > ta) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tc_ld16(tO + c, o);
                        tc_wait_ld();
                        tc_regs_ready(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc_st16(tO + c, o);
                    }
                }
                const float neg = m == -INFINITY ? 0.0f : -m;
                const uint64_t scale2 = pair2(p.scale_log2, p.scale_log2), neg2 = pair2(neg, neg);
                uint64_t s0 = 0, s1 = 0;
#pragma unroll
                for (int b = 0; b < 128; b += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        float a0, a1, a2, a3;
                        split2(a0, a1, fma2(pair2(__uint_as_float(v[b + c]), __uint_as_float(v[b + c + 1])), scale2, neg2));
                        split2(a2, a3, fma2(pair2(__uint_as_float(v[b + c + 2]), __uint_as_float(v[b + c + 3])), scale2, neg2));
                        a0 = ex2(a0);
                        a1 = ex2(a1);
                        a2 = ex2(a2);
                        a3 = ex2(a3);
                        s0 = add2(s0, pair2(a0, a1));
                        s1 = add2(s1, pair2(a2, a3));
                        pk[c / 2] = pack16<BF16>(a0, a1);
                        pk[c / 2 + 1] = pack16<BF16>(a2, a3);
                    }
                    tc_st16(tS + b / 2, pk);
                }
                float l0, l1;
                split2(l0, l1, add2(s0, s1));
                l += l0 + l1;
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[i]);
            }
            // ---- results
            const bool has = tb > ta;
            if (has) mbar_wait(&ofull[i], 0, p.err, &abort_flag, lim);
            tc_fence_after();
            float lse;
            const float f = softmax_finish(m, l, p.sinks != nullptr, p.sinks ? p.sinks[head] * 1.4426950408889634f : 0.0f, lse);
            const bool mine = row < w.rows;
            const uint64_t orow = (uint64_t)(w.q0 + w.row0 + row) * p.n_heads + head;
            const bool fix = dirty != 0;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tc_ld32(tO + c, o);
                tc_wait_ld();
                tc_regs_ready(o);
                float y[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = f == 0.0f ? 0.0f : __uint_as_float(o[e]) * f;
                if (mine) {
                    if (fix) {
                        const uint16_t *vp = static_cast<const uint16_t *>(p.v) + (uint64_t)w.k0 * p.v_stride + (uint64_t)kvh * D + c;
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            float z[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) z[k] = y[e + k];
                            prompt_restore<BF16>(p, w, vp + e, row, C::BN, z);
#pragma unroll
                            for (int k = 0; k < 8; ++k) y[e + k] = z[k];
                        }
                    }
                    store_row32(p, orow, c, y);
                }
            }
            if (p.lse && mine) p.lse[orow] = lse;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <int D, bool BF16> cudaError_t launch_tc(const AttnPromptParams &p, cudaStream_t st) {
    static bool attr_done = false;
    if (!attr_done) {
        const cudaError_t e = cudaFuncSetAttribute(k_attn_prompt_tc<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   Pt<D>::SMEM);
        if (e != cudaSuccess) return e;
        attr_done = true;
    }
    alignas(64) CUtensorMap tmQ, tmK, tmV;
    if (!encode_rows16_tmap(&tmQ, p.q, (uint64_t)p.n_heads * D, p.n_q, p.q_stride, 128, BF16) ||
        !encode_rows16_tmap(&tmK, p.k, (uint64_t)p.n_kv * D, p.n_k, p.k_stride, 128, BF16) ||
        !encode_rows16_tmap(&tmV, p.v, (uint64_t)p.n_kv * D, p.n_k, p.v_stride, 128, BF16))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.n_heads, p.n_q / Pt<D>::BM + p.n_seq);   // heads of one tile side by side, long tiles first
    cfg.blockDim = dim3(Pt<D>::THREADS);
    cfg.dynamicSmemBytes = Pt<D>::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_attn_prompt_tc<D, BF16>, p, tmQ, tmK, tmV);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_attn_prompt_tc(const AttnPromptParams &p, cudaStream_t st) {
    const bool bf = p.type == Q8_TYPE_BF16;
    if (p.dim == 64) return bf ? launch_tc<64, true>(p, st) : launch_tc<64, false>(p, st);
    return bf ? launch_tc<128, true>(p, st) : launch_tc<128, false>(p, st);
}

}  // namespace q8
