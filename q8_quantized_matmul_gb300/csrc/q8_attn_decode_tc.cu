// q8_attn_decode_tc.cu -- decode attention on the 5th-generation tensor cores, for large heads (256 or 512
// values, 16 bit) that more than 16 query heads share: q_b's 64 heads of 512 on one key-value head.
//
// The mma.sync kernel would read the cache once per 16 heads there and is bound by its products (64 heads
// cost 64 operations a cached byte).  Here a unit is (sequence, key-value head, 64 of its query heads) and a
// step is 128 positions, both products transposed so that no row of a tile is idle:
//   S^T [128 positions x 64 heads]  = K Q^T     A: K tile, B: Q, both K-major; D / 16 UMMAs of N = 64
//   O^T [D dims x 64 heads]        += V^T P^T   A: V tile as it lies (M contiguous), B: P; D / 128 M tiles
// in TMEM columns 0-63 and 64 + 64 i.  One thread per position reads its 64 scores, writes P as a row of 64
// 16-bit weights to shared memory and keeps its own sums l[64].  The running maximum of a head is moved
// only when a score exceeds it by more than 2^8 (one vote a step); then the maxima are reduced and O^T, l
// rescaled.  Cached bytes enter once through a ring of 32 KB slots (128 positions x 128 dims, by TMA page by
// page, K and V in turn), 128 KB in flight.  16 sequences of up to 4100 positions take 26 us, three times the bytes'
// time: with 1.4 steps a CTA the start (256 KB a CTA) and the pieces set it, not the stream.
//
// The line of steps is cut into equal shares as in the mma.sync kernel.  A CTA that has all of a unit writes its
// result (200 sequences of 16 positions: 48.8 -> 30.5 us); of a unit that is cut every share leaves its (m, l, O) in scratch (a
// unit's 128 KB would take one CTA 10 us to join) and k_attn_decode_join adds them, two heads a CTA, in order.  Only the
// first and the last unit of a share can be cut, so each CTA has two places there.
//
// Positions that are not visible are masked in S; their V rows are set to zero in shared memory before the
// product (guard warps), whatever the page holds there.  Waits are bounded as everywhere.
#include "q8_attn.cuh"
#include "q8_attn_decode.cuh"
#include "q8_kv.h"
#include "q8_launch.h"
#include "q8_tcgen05.cuh"

namespace q8 {

bool encode_3d16_tmap(CUtensorMap *map, const void *base, uint64_t cols, uint64_t n1, uint64_t n2, uint64_t stride1,
                      uint64_t stride2, uint32_t box1, uint32_t box2, bool bf16);

namespace {

template <int D> struct Dt {
    static constexpr int HT = 64, TT = 128;                  // heads of a unit, positions of a step
    static constexpr int KS = D / 128;                       // slots of a K (or V) tile
    static constexpr int CHUNK = 128 * 128;                  // 128 positions x 64 dims
    static constexpr int SLOT = 2 * CHUNK, NST = 4;
    static constexpr int QBYTES = HT * D * 2, PBYTES = TT * HT * 2;
    static constexpr int THREADS = 256;
    static constexpr int NBAR = 2 + 3 * NST + 3 + 1;
    static constexpr int FLOATS = HT * (1 + 1 + 1 + 4);      // m, references, factors, per-warp maxima
    static constexpr int SMEM = 1024 + QBYTES + PBYTES + NST * SLOT + NBAR * 8 + FLOATS * 4 + 64;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ bool warps_any(bool v) {          // over the four softmax warps
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

// Reduces 64 values a lane over the warp's 32 lanes: lane i ends with the results of 2 i and 2 i + 1.
template <class F> __device__ __forceinline__ void reduce64(float (&v)[64], F f) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = 32, b = 16; b; w >>= 1, b >>= 1) {
        const bool up = lane & b;                            // keeps the upper half of what is left
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float give = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
            v[i] = f(keep, __shfl_xor_sync(0xffffffffu, give, b));
        }
    }
}

struct Line {                                                // a CTA's share of the line
    int64_t total, t0, t1, s_base;
    uint32_t s, shares;
    int run;                                                 // steps of an element of the line
};

// A lane's value of the Q8_0 block that the warp's 32 lanes hold.
__device__ __noinline__ void store_q8_lane(uint8_t *blk, float y) {
    const int lane = threadIdx.x & 31;
    const float d = __fdiv_rn(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fabsf(y), 0.0f)))), 127.0f);
    blk[2 + lane] = (uint8_t)(d != 0.0f ? (int)roundf(__fdiv_rn(y, d)) : 0);
    if (lane == 0) *reinterpret_cast<uint16_t *>(blk) = d != 0.0f ? __half_as_ushort(__float2half_rn(d)) : 0;
}

// One dim (this thread's) of `n` of 32 heads, times each head's factor (0: nothing seen), as results; i0: place of the first,
// the next heads' lie D on.  The type is asked for once: asked for each value, a unit took 40 us to write, not 3.
template <int D>
__device__ __forceinline__ void store_dim(const AttnDecodeParams &p, uint64_t i0, int n, const uint32_t (&o)[32], const float *factor) {
    float y[32];
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        const float4 f4 = *reinterpret_cast<const float4 *>(factor + e);
        const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) y[e + k] = f[k] == 0.0f ? 0.0f : __uint_as_float(o[e + k]) * f[k];
    }
    if (p.out_type == Q8_TYPE_Q8_0) {
        uint8_t *blk = static_cast<uint8_t *>(p.out) + i0 / QK * QB;
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (e < n) store_q8_lane(blk + (size_t)e * (D / QK * QB), y[e]);
    } else if (p.out_type == Q8_TYPE_F32) {
        float *dst = static_cast<float *>(p.out) + i0;
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (e < n) dst[(size_t)e * D] = y[e];
    } else {
        uint16_t *dst = static_cast<uint16_t *>(p.out) + i0;
        const bool bf = p.out_type == Q8_TYPE_BF16;
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) w[e / 2] = bf ? pack16<true>(y[e], y[e + 1]) : pack16<false>(y[e], y[e + 1]);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (e < n) dst[(size_t)e * D] = (uint16_t)(w[e / 2] >> (e % 2 * 16));
    }
}

// The segment (part of one unit) that starts at element `at` of the line.
struct Segment64 {
    Seq q;
    uint32_t s, kvh, head0, unit_id;
    int rows, ta, tb;                                        // steps [ta, tb)
    int64_t u0, next;                                        // the unit's first element; the one after the segment
    int elements;                                            // of the unit
};

template <int D, bool BF16>
__global__ void __launch_bounds__(Dt<D>::THREADS, 1)
    k_attn_decode_tc(const AttnDecodeParams p, const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
    using C = Dt<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    __shared__ volatile uint32_t pieces_ok[2];               // step n & 1: pieces that have a page
    __shared__ int64_t scan[10 + C::THREADS / 32];
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *qs = smem, *ps = qs + C::QBYTES, *ring = ps + C::PBYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + C::NST * C::SLOT);
    uint64_t *qfull = bars, *qempty = bars + 1, *full = bars + 2, *empty = full + C::NST, *ready = empty + C::NST;
    uint64_t *sfull = ready + C::NST, *pfull = sfull + 1, *ofull = pfull + 1, *done = ofull + 1;
    float *sm_m = reinterpret_cast<float *>(bars + C::NBAR), *sm_r = sm_m + C::HT, *sm_f = sm_r + C::HT,
          *sm_w = sm_f + C::HT;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint64_t lim = wait_limit(p.wait_ns);

    if (tid == 0) {
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        for (int i = 0; i < C::NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&ready[i], 2);
        }
        mbar_init(sfull, 1);
        mbar_init(pfull, 4);
        mbar_init(ofull, 1);
        mbar_init(done, 1);
        abort_flag = 0;
        fence_mbar_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmQ)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmK)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmV)) : "memory");
    }
    grid_dep_wait();
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const int box = min(1 << p.c.page_shift, 128), box_shift = min((int)p.c.page_shift, 7);
    const uint32_t units_per_seq = p.c.n_kv * p.mtiles;

    // ---- this CTA's share of the line, and the sequence it starts in.  A piece costs 128 KB of writes and reads
    // however short it is: with at most half as many units as CTAs the line's elements are runs of steps that
    // give no CTA more than one piece (16 sequences of up to 4100 positions: 31.7 -> 29.2 us), else single steps.
    Line L;
    {
        const uint32_t per = (p.n_seq + C::THREADS - 1) / C::THREADS, a = min(p.n_seq, tid * per), b = min(p.n_seq, a + per);
        auto prefix = [&](int run, bool raise, int64_t &mine, int64_t &before, int64_t &total, int64_t &units) {
            mine = 0;
            int64_t used = 0;
#pragma unroll 8
            for (uint32_t i = a; i < b; ++i) {
                const int n = seq_of(C::TT, box, p, i, raise).tiles;
                mine += (n + run - 1) / run;
                used += n > 0;
            }
            mine *= units_per_seq;
            int64_t sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) used += __shfl_xor_sync(0xffffffffu, used, o);
            if (lane == 31) {
                scan[warp] = sum;
                scan[10 + warp] = used;
            }
            __syncthreads();
            before = sum - mine;
            total = units = 0;
            for (int w = 0; w < C::THREADS / 32; ++w) {
                if (w < warp) before += scan[w];
                total += scan[w];
                units += scan[10 + w];
            }
            units *= units_per_seq;
            __syncthreads();
        };
        int64_t mine, before, units;
        prefix(1, blockIdx.x == 0, mine, before, L.total, units);
        L.run = 1;
        if (units > 0 && 2 * units <= (int64_t)gridDim.x) {
            // sum of ceil(n / run) <= total / run + units <= CTAs
            const int64_t room = (int64_t)gridDim.x - units;
            L.run = (int)min((L.total + room - 1) / room, (int64_t)1 << 24);
            if (L.run > 1) prefix(L.run, false, mine, before, L.total, units);
        }
        L.shares = L.total < (int64_t)gridDim.x ? (uint32_t)L.total : gridDim.x;   // every share has an element
        L.t0 = L.t1 = 0;
        if (blockIdx.x < L.shares) {
            L.t0 = L.total * blockIdx.x / L.shares;
            L.t1 = L.total * (blockIdx.x + 1) / L.shares;
        }
        if (L.t0 < L.t1 && before <= L.t0 && L.t0 < before + mine) {
            uint32_t i = a;
            for (;; ++i) {
                const int64_t n = (int64_t)((seq_of(C::TT, box, p, i, false).tiles + L.run - 1) / L.run) * units_per_seq;
                if (L.t0 < before + n) break;
                before += n;
            }
            scan[8] = i;
            scan[9] = before;
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        L.s = (uint32_t)scan[8];
        L.s_base = scan[9];
    }
    const uint32_t tmem = tmem_slot;
    auto segment = [&](int64_t at, Line &w) {                // w.s, w.s_base move forward
        Segment64 g;
        g.q = seq_of(C::TT, box, p, w.s, false);
        g.elements = (g.q.tiles + w.run - 1) / w.run;
        while (at >= w.s_base + (int64_t)g.elements * units_per_seq) {
            w.s_base += (int64_t)g.elements * units_per_seq;
            g.q = seq_of(C::TT, box, p, ++w.s, false);
            g.elements = (g.q.tiles + w.run - 1) / w.run;
        }
        const uint32_t unit = (uint32_t)((at - w.s_base) / g.elements);
        g.u0 = w.s_base + (int64_t)unit * g.elements;
        g.next = min(g.u0 + g.elements, w.t1);
        g.ta = (int)(at - g.u0) * w.run;
        g.tb = (int)min((int64_t)g.q.tiles, (g.next - g.u0) * w.run);
        g.s = w.s;
        g.kvh = unit / p.mtiles;
        const uint32_t mt = unit % p.mtiles;
        g.head0 = g.kvh * p.group + mt * C::HT;
        g.rows = (int)min((uint32_t)C::HT, p.group - mt * C::HT);
        g.unit_id = w.s * units_per_seq + unit;
        return g;
    };

    // ---- sequences with nothing visible have no pieces
    for (uint64_t i = (uint64_t)blockIdx.x * C::THREADS + tid; i < (uint64_t)p.n_seq * units_per_seq; i += (uint64_t)gridDim.x * C::THREADS)
        if (seq_of(C::TT, box, p, (uint32_t)(i / units_per_seq), false).tiles == 0) p.units[i] = make_int4(0, 0, 0, 0);

    Line w = L;
    if (warp == 4) {
        // ------------------------------------------------ TMA producer: lane j the j-th piece of a page
        uint32_t fills[C::NST] = {}, q_loads = 0, u = 0, n = 0;
        auto go = [&](uint64_t *bar, uint32_t parity) {
            return __shfl_sync(0xffffffffu, (int)(!p.withhold && tile_wait(bar, parity, p.err, &abort_flag, lim) && !abort_flag), 0) != 0;
        };
        for (int64_t at = L.t0; at < L.t1;) {
            const Segment64 g = segment(at, w);
            if (go(qempty, (q_loads & 1) ^ 1)) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(qfull, C::QBYTES);
                    for (int c = 0; c < D / 64; ++c)
                        tma_load_3d(qs + c * C::HT * 128, &tmQ, 64 * c, (int)g.head0, (int)g.s, qfull);
                }
                ++q_loads;
            }
            __syncwarp();
            const int32_t *pages = p.table + (uint64_t)g.s * p.table_stride;
            const int n_pc = 128 >> box_shift;
            for (int it = g.ta; it < g.tb; ++it, ++n) {
                const int pos = g.q.start + it * C::TT + lane * box;
                int page = -1;
                if (lane < n_pc && pos < g.q.hi) {
                    page = pages[pos >> p.c.page_shift];
                    if (page < 0 || (uint32_t)page >= p.c.n_pages) {
                        raise_error(p.err, DEV_ERANGE);
                        page = -1;
                    }
                }
                const uint32_t okm = __ballot_sync(0xffffffffu, page >= 0);
                const uint32_t bytes = __popc(okm) * box * 128 * 2;
                const int y = (int)g.kvh << p.c.page_shift | (pos & ((1 << p.c.page_shift) - 1));
                for (int j = 0; j < 2 * C::KS; ++j, ++u) {   // slots of K, then of V
                    const int st = u % C::NST;
                    if (go(&empty[st], ((u / C::NST) & 1) ^ 1)) {
                        if (lane == 0) {
                            pieces_ok[n & 1] = okm;
                            if (bytes) mbar_arrive_expect_tx(&full[st], bytes);
                            else mbar_arrive(&full[st]);
                        }
                        __syncwarp();
                        if (page >= 0) {
                            uint8_t *t = ring + st * C::SLOT + lane * box * 128;
                            const CUtensorMap *map = j < C::KS ? &tmK : &tmV;
                            for (int c = 0; c < 2; ++c)
                                tma_load_3d(t + c * C::CHUNK, map, (j % C::KS * 2 + c) * 64, y, page, &full[st]);
                        }
                        ++fills[st];
                    }
                    __syncwarp();
                }
            }
            at = g.next;
        }
        if (abort_flag && lane == 0) {
            const uint64_t t_end = global_timer_ns() + WAIT_LIMIT_NS;
            if (q_loads) mbar_drain(qfull, (q_loads - 1u) & 1u, t_end);
            for (int s = 0; s < C::NST; ++s)
                if (fills[s]) mbar_drain(&full[s], (fills[s] - 1u) & 1u, t_end);
        }
        __syncwarp();
    } else if (warp == 5) {
        // ------------------------------------------------ UMMA issuer
        constexpr uint32_t idS = tc_idesc(128, C::HT, BF16), idO = tc_idesc(128, C::HT, BF16, true, true);
        const uint64_t dq = sw128_desc(smem_addr(qs)), dk = sw128_desc(smem_addr(ring)),
                       dv = sw128_desc_mn(smem_addr(ring), C::CHUNK), dp = sw128_desc_mn(smem_addr(ps), C::CHUNK);
        bool ok = true;
        uint32_t u = 0, n = 0, q_loads = 0;
        for (int64_t at = L.t0; at < L.t1;) {
            const Segment64 g = segment(at, w);
            ok = tile_wait(qfull, q_loads & 1, p.err, &abort_flag, lim) && ok;
            ++q_loads;
            for (int it = g.ta; it < g.tb; ++it, ++n) {
                for (int j = 0; j < C::KS; ++j, ++u) {
                    const int st = u % C::NST;
                    ok = tile_wait(&ready[st], (u / C::NST) & 1, p.err, &abort_flag, lim) && ok;
                    tc_fence_after();
                    if (elect_one()) {
                        if (ok) {
                            const uint64_t a = dk + (uint32_t)st * (C::SLOT / 16), b = dq + (uint32_t)j * (2 * C::HT * 128 / 16);
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                tc_mma_f16(tmem, a + (k / 4) * (C::CHUNK / 16) + (k % 4) * 2, b + (k / 4) * (C::HT * 128 / 16) + (k % 4) * 2,
                                           idS, j > 0 || k > 0);
                            tc_commit(&empty[st]);
                        }
                        if (j == C::KS - 1) {
                            tc_commit(sfull);
                            if (it == g.tb - 1 && ok) tc_commit(qempty);
                        }
                    }
                    __syncwarp();
                }
                ok = tile_wait(pfull, n & 1, p.err, &abort_flag, lim) && ok;
                for (int j = 0; j < C::KS; ++j, ++u) {
                    const int st = u % C::NST;
                    ok = tile_wait(&ready[st], (u / C::NST) & 1, p.err, &abort_flag, lim) && ok;
                    tc_fence_after();
                    if (elect_one()) {
                        if (ok) {
                            const uint64_t a = dv + (uint32_t)st * (C::SLOT / 16);
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                tc_mma_f16(tmem + 64 + j * 64, a + k * (2048 / 16), dp + k * (2048 / 16), idO, it > g.ta || k > 0);
                            tc_commit(&empty[st]);
                        }
                        if (j == C::KS - 1 && it == g.tb - 1) tc_commit(ofull);
                    }
                    __syncwarp();
                }
            }
            at = g.next;
        }
        if (elect_one()) tc_commit(done);
        __syncwarp();
        tile_wait(done, 0, p.err, nullptr);   // the fixed 2 s limit: TMEM is freed after this
    } else if (warp >= 6) {
        // ------------------------------------------------ V guard: two threads a position's row
        const int gt = tid - 192;
        uint32_t u = 0, n = 0;
        for (int64_t at = L.t0; at < L.t1;) {
            const Segment64 g = segment(at, w);
            for (int it = g.ta; it < g.tb; ++it, ++n)
                for (int j = 0; j < 2 * C::KS; ++j, ++u) {
                    const int st = u % C::NST;
                    const bool ok = tile_wait(&full[st], (u / C::NST) & 1, p.err, &abort_flag, lim);
                    if (ok && j >= C::KS) {
                        const int p0 = g.q.start + it * C::TT;
                        const uint32_t okm = pieces_ok[n & 1], all = (2u << ((128 >> box_shift) - 1)) - 1u;
                        if (p0 < g.q.lo || p0 + C::TT > g.q.hi || okm != all) {
                            uint8_t *t = ring + st * C::SLOT;
                            for (int r = gt >> 1; r < 128; r += 32) {
                                const int pos = p0 + r;
                                if (pos >= g.q.lo && pos < g.q.hi && ((okm >> (r >> box_shift)) & 1)) continue;
                                uint4 *row = reinterpret_cast<uint4 *>(t + (gt & 1) * C::CHUNK + r * 128);
#pragma unroll
                                for (int e = 0; e < 8; ++e) row[(e + r) & 7] = make_uint4(0, 0, 0, 0);   // rows 128 bytes apart: other banks
                            }
                            fence_async_smem();
                        }
                    }
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(&ready[st]);
                }
            at = g.next;
        }
    } else {
        // ------------------------------------------------ softmax, one position a thread; then O^T, one dim a thread
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const int r = tid;                                   // position within the step
        uint8_t *prow = ps + r * 128;
        uint32_t n = 0, o_seen = 0;
        bool first = true;
        for (int64_t at = L.t0; at < L.t1; first = false) {
            const Segment64 g = segment(at, w);
            float l[64];
#pragma unroll
            for (int h = 0; h < 64; ++h) l[h] = 0.0f;
            if (tid < 64) {
                sm_m[tid] = -INFINITY;
                sm_r[tid] = 0.0f;                            // 2^(-inf - 0): a head that has seen nothing has no weights
            }
            named_bar_sync(2, 128);
            for (int it = g.ta; it < g.tb; ++it, ++n) {
                tile_wait(sfull, n & 1, p.err, &abort_flag, lim);
                tc_fence_after();
                const int pos = g.q.start + it * C::TT + r;
                const bool seen = pos >= g.q.lo && pos < g.q.hi && ((pieces_ok[n & 1] >> (r >> box_shift)) & 1);
                uint32_t v[64];
                tc_ld32(tmem + lanes, v);
                tc_ld32(tmem + lanes + 32, v + 32);
                tc_wait_ld();
                tc_regs_ready(v);
                float z[64];
                bool grow = false;
#pragma unroll
                for (int h = 0; h < 64; h += 4) {
                    const float4 m4 = *reinterpret_cast<const float4 *>(sm_m + h);
                    const float mm[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        z[h + e] = seen ? __uint_as_float(v[h + e]) * p.scale_log2 : -INFINITY;
                        grow |= z[h + e] > mm[e] + 8.0f;
                    }
                }
                if (warps_any(grow)) {
                    float x[64];
#pragma unroll
                    for (int h = 0; h < 64; ++h) x[h] = z[h];
                    reduce64(x, [](float a, float b) { return fmaxf(a, b); });
                    sm_w[warp * 64 + 2 * lane] = x[0];
                    sm_w[warp * 64 + 2 * lane + 1] = x[1];
                    named_bar_sync(2, 128);
                    if (tid < 64) {
                        const float old = sm_m[tid];
                        const float mx = fmaxf(fmaxf(sm_w[tid], sm_w[64 + tid]), fmaxf(sm_w[128 + tid], sm_w[192 + tid]));
                        const float now = mx > old + 8.0f ? mx : old;
                        sm_m[tid] = now;
                        sm_r[tid] = now == -INFINITY ? 0.0f : weight_ref<LAZY_UP<BF16>>(now);
                        // a first maximum: nothing to rescale
                        sm_f[tid] = old == now || old == -INFINITY ? 1.0f : ex2(weight_ref<LAZY_UP<BF16>>(old) - weight_ref<LAZY_UP<BF16>>(now));
                    }
                    named_bar_sync(2, 128);
                    if (it > g.ta) {
#pragma unroll
                        for (int h = 0; h < 64; ++h) l[h] *= sm_f[h];
#pragma unroll 1
                        for (int c = 0; c < D / 128 * 64; c += 16) {
                            uint32_t o[16];
                            tc_ld16(tmem + lanes + 64 + c, o);
                            tc_wait_ld();
                            tc_regs_ready(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * sm_f[(c & 63) + e]);
                            tc_st16(tmem + lanes + 64 + c, o);
                        }
                        tc_wait_st();
                    }
                }
                uint32_t pk[32];
#pragma unroll
                for (int h = 0; h < 64; h += 4) {
                    const float4 r4 = *reinterpret_cast<const float4 *>(sm_r + h);
                    const float rr[4] = {r4.x, r4.y, r4.z, r4.w};
                    float a[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        a[e] = ex2(z[h + e] - rr[e]);
                        l[h + e] += a[e];
                    }
                    pk[h / 2] = pack16<BF16>(a[0], a[1]);
                    pk[h / 2 + 1] = pack16<BF16>(a[2], a[3]);
                }
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    *reinterpret_cast<uint4 *>(prow + ((c ^ (r & 7)) << 4)) = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull);
            }
            // ---- sums over the positions, then O^T: the unit's result, or this share's piece as it stands
            tile_wait(ofull, o_seen & 1, p.err, &abort_flag, lim);
            ++o_seen;
            tc_fence_after();
            reduce64(l, [](float a, float b) { return a + b; });
            named_bar_sync(2, 128);                          // sm_w is free
            sm_w[warp * 64 + 2 * lane] = l[0];
            sm_w[warp * 64 + 2 * lane + 1] = l[1];
            named_bar_sync(2, 128);
            const uint64_t slot = 2 * (uint64_t)blockIdx.x + (first ? 0 : 1);
            // (A line of runs gives a CTA one piece at most, and a piece leaves sooner than a result: 16 sequences of up to 4100
            // positions 27.1 -> 26.3 us.)
            const bool whole = g.ta == 0 && g.tb == g.q.tiles && L.run == 1;
            if (tid < 64) {
                const float m = weight_ref<LAZY_UP<BF16>>(sm_m[tid]), sum = (sm_w[tid] + sm_w[64 + tid]) + (sm_w[128 + tid] + sm_w[192 + tid]);
                if (whole) {
                    const bool act = tid < g.rows;
                    float lse;
                    sm_f[tid] = softmax_finish(m, sum, p.sinks != nullptr, sink_of(p, g.head0 + tid, act), lse);
                    if (act && p.lse) p.lse[(uint64_t)g.s * p.n_heads + g.head0 + tid] = lse;
                } else {
                    p.part_ml[slot * 64 + tid] = make_float2(m, sum);
                }
            }
            if (!whole) {
#pragma unroll 1
                for (int c = 0; c < D / 128 * 64; c += 32) {
                    uint32_t o[32];
                    tc_ld32(tmem + lanes + 64 + c, o);
                    tc_wait_ld();
                    tc_regs_ready(o);
                    float *dst = p.part + (slot * 64 + (c & 63)) * D + (c >> 6) * 128 + r;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if ((c & 63) + e < g.rows) dst[(uint64_t)e * D] = __uint_as_float(o[e]);
                }
            } else {
                named_bar_sync(2, 128);                      // the factors
#pragma unroll 1
                for (int c = 0; c < D / 128 * 64; c += 32) {
                    uint32_t o[32];
                    tc_ld32(tmem + lanes + 64 + c, o);
                    tc_wait_ld();
                    tc_regs_ready(o);
                    const int h0 = c & 63, d = (c >> 6) * 128 + r;
                    store_dim<D>(p, ((uint64_t)g.s * p.n_heads + g.head0 + h0) * D + d, g.rows - h0, o, sm_f + h0);
                }
            }
            tc_fence_before();
            if (whole && tid == 0) {
                p.units[g.unit_id] = make_int4(0, 0, -1, 0); // nothing to join
            } else if (g.ta == 0 && tid == 0) {
                // the unit starts here: where its pieces are (the first in this CTA, the others each CTA's first)
                int64_t last = (g.u0 + g.elements - 1) * L.shares / L.total;
                while (L.total * (last + 1) / L.shares <= g.u0 + g.elements - 1) ++last;
                while (L.total * last / L.shares > g.u0 + g.elements - 1) --last;
                p.units[g.unit_id] = make_int4((int)slot, (int)blockIdx.x, (int)(last - blockIdx.x) + 1, 0);
            }
            named_bar_sync(2, 128);                          // sm_m, sm_w are read
            at = g.next;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// out = sum of the pieces: D / 8 threads a head, 128 threads a CTA.
template <int D> __global__ void __launch_bounds__(128) k_attn_decode_join(const AttnDecodeParams p) {
    grid_dep_wait();
    constexpr int TH = D / 8;
    const uint64_t item = (uint64_t)blockIdx.x * (128 / TH) + threadIdx.x / TH;
    const bool act = item < (uint64_t)p.n_seq * p.n_heads;
    const uint32_t s = act ? (uint32_t)(item / p.n_heads) : 0, head = act ? (uint32_t)(item % p.n_heads) : 0;
    const uint32_t kvh = head / p.group, mt = head % p.group / 64, row = head % p.group % 64;
    const int d0 = threadIdx.x % TH * 8;
    const int4 un = p.units[((uint64_t)s * p.c.n_kv + kvh) * p.mtiles + mt];
    auto slot_of = [&](int k) { return k == 0 ? (uint64_t)un.x : 2 * (uint64_t)(un.y + k); };
    const float sink = sink_of(p, head, act);
    if (un.z < 0) return;                                    // written by the CTA that had all of it (the whole warp)
    float m, l, y[8];
    join8(un.z, [&](int k) { return p.part + (slot_of(k) * 64 + row) * D + d0; },
          [&](int k) { return p.part_ml + slot_of(k) * 64 + row; }, m, l, y);
    finish8(p, s, head, d0, sink, m, l, y, act);
}

template <int D, bool BF16> cudaError_t launch_tc(const AttnDecodeParams &p, int grid, cudaStream_t st) {
    static SmemAllowed allowed;
    const cudaError_t es = allow_smem(allowed, reinterpret_cast<const void *>(k_attn_decode_tc<D, BF16>), Dt<D>::SMEM);
    if (es != cudaSuccess) return es;
    alignas(64) CUtensorMap tmQ, tmK, tmV;
    const uint32_t tokens = 1u << p.c.page_shift, box = tokens < 128 ? tokens : 128;
    if (!encode_3d16_tmap(&tmQ, p.q, D, p.n_heads, p.n_seq, D, p.q_stride, Dt<D>::HT, 1, BF16) ||
        !encode_3d16_tmap(&tmK, p.c.k, D, (uint64_t)p.c.n_kv * tokens, p.c.n_pages, D, p.c.page_stride / 2, box, 1, BF16) ||
        !encode_3d16_tmap(&tmV, p.c.v, D, (uint64_t)p.c.n_kv * tokens, p.c.n_pages, D, p.c.page_stride / 2, box, 1, BF16))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(Dt<D>::THREADS);
    cfg.dynamicSmemBytes = Dt<D>::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, k_attn_decode_tc<D, BF16>, p, tmQ, tmK, tmV);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const uint64_t per = 128 / (D / 8), ctas = ((uint64_t)p.n_seq * p.n_heads + per - 1) / per;
    return launch_dependent(k_attn_decode_join<D>, p, dim3((unsigned)ctas), 128, 0, st);
}

}  // namespace

cudaError_t launch_attn_decode_tc(const AttnDecodeParams &p, int grid, cudaStream_t st) {
    const bool bf = p.q_type == Q8_TYPE_BF16;
    if (p.c.dim == 256) return bf ? launch_tc<256, true>(p, grid, st) : launch_tc<256, false>(p, grid, st);
    return bf ? launch_tc<512, true>(p, grid, st) : launch_tc<512, false>(p, grid, st);
}

}  // namespace q8
