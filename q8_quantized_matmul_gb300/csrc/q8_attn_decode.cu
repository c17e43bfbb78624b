// q8_attn_decode.cu -- attention of one new token per sequence over a paged cache.
//
//   z_j = scale q.k_j,  out = sum_j 2^(z_j - m) v_j / (sum_j 2^(z_j - m) + 2^(sink - m))   (z in log2 units)
//
// One pass over the visible positions with a running maximum m, sum l and unnormalised output O
// (all fp32).  Every cached byte is read once, so HBM is the bound: 2 D values per position and
// key-value head against 4 D operations per query head.  48 sequences of up to 16 000 positions, 8 key-value heads of
// 128 in bf16: 111 us, 6.2 TB/s (0.92 of a copy's rate); 4 of up to 100 003 in Q8_0: 61.4 us, 5.2 TB/s, with the
// conversion of the quants on the ALU at half its rate.
//
// Split.  A unit is (sequence, key-value head, tile of 8 or 16 of its query heads).  The products run
// transposed, positions (scores) and V dimensions (output) along the 16 rows of an mma.sync tile and the
// heads that share K and V along its 8 columns: groups of up to 8 heads waste no rows, and the accumulators
// of 8 heads by 128 dimensions take 32 registers.  P goes from one product's layout to the other's by
// movmatrix.  The units' positions, in tiles of TT, form one line that is cut into equal shares, one per
// CTA, so the lengths do not matter to the balance.  A CTA that covers a whole unit writes its result;
// otherwise it leaves (m, l, O) in scratch, and the last CTA of a unit to arrive (one counter per unit, set
// back to zero by it) joins the pieces in their order: the same bits on every run.  A unit of many pieces is
// joined in two steps, so that no CTA reads hundreds of them one round after another.
//
// Inside a CTA each of the four warps takes its own 16 (Q8_0: 32) positions of a tile through its own
// ring of stages, filled by 16-byte asynchronous copies, and keeps its own (m, l, O): no CTA barrier
// until the unit's share ends.  A head of 512 values does not fit a warp's registers as O, so there
// two warps share the positions and own half of V's dimensions each.
// Rows that are not visible (other positions of the first or last page, a page id outside the pool)
// are filled with zeros and masked, so whatever they hold never reaches a product.
//
// Q8_0 pages: int8 quants are exact in either 16-bit type.  The score sums each 32-value block on its
// own and folds the block's K scale in fp32, exact but for fp32 rounding.  V's scale goes into the
// weights, one fp16 rounding each: 2^(z - M + 15) d with M >= m + e, every |d| < 2^e of the slice, so
// products stay below 2^15 and the weights keep 29 binades above the smallest normal.  The weights of fp16 caches are
// 2^(z - m + 15) for the same reason.
#include <algorithm>

#include "q8_attn.cuh"
#include "q8_attn_decode.cuh"
#include "q8_kv.h"
#include "q8_launch.h"

namespace q8 {
namespace {

// Pieces that one CTA joins at once, and in groups when there are more (24 pieces a unit: in groups 12.1 us, at once 10.7;
// 30: 12.4 and 13.6; 228: 21 and 68).
constexpr int AT_ONCE = 24, GROUP = 16;
// Tiles of the line before each unit's first that hold nothing: a CTA that works on two units pays for the second start
// with fewer tiles (24 units over 608 CTAs: 16.8 -> 14.0 us; 60 Q8_0 units over 304: 27.8 -> 24.4; 32 long ones: 63.4 ->
// 61.8; 8 and 16 tiles gain on few units and lose on many).
constexpr int HEAD = 2;

// FMT 0: f16, 1: bf16, 2: Q8_0 with f16 q, 3: Q8_0 with bf16 q; NT tiles of 8 heads a unit
template <int D, int FMT, int NT> struct Dec {
    static constexpr bool Q8 = FMT >= 2, BF16 = FMT & 1;
    static constexpr int HR = 8 * NT;                    // heads of a unit
    static constexpr int W = 4;                          // warps
    static constexpr int ST = Q8 ? 32 : 16;              // positions of a warp's slice
    static constexpr int DV = D > 256 ? 256 : D;         // V dimensions of a warp
    static constexpr int NDH = D / DV;                   // warps that share a slice
    static constexpr int SL = W / NDH;                   // slices in a tile
    static constexpr int TT = SL * ST;                   // positions of a tile
    static constexpr int KB = ST * D * (Q8 ? 1 : 2), VB = ST * DV * (Q8 ? 1 : 2);
    static constexpr int KSB = Q8 ? ST * (D / 32) * 2 : 0, VSB = Q8 ? ST * (DV / 32) * 2 : 0;
    static constexpr int STAGE = KB + VB + KSB + VSB;
    // When no sequence has more tiles than this, CTAs take whole units: joining pieces costs 2 to 3 us (heads of 512: 6
    // to 9), as much as these tiles one after another.  One sequence of t tiles, 8 or 16 heads a unit, pieces / whole units, us:
    //   16 bit:  64 values t = 8 6.6 / 6.5, 10 7.3 / 7.4;  128 t = 5 7.0 / 6.6, 6 7.0 / 7.3;  256 t = 4 9.5 / 8.6, 5 9.7 / 9.8;
    //            512 t = 5 12.4 / 12.7, 16 heads 18.8 / 16.0
    //   Q8_0:    64 values t = 4 7.4 / 6.6, 5 7.6 / 7.6;  128 t = 3 8.5 / 7.9, 4 8.5 / 9.2;  256 t = 2 10.9 / 11.1, 5 12.4 / 21.9;
    //            512 t = 2 17.0 / 16.0, 3 16.9 / 21.4
    // (16 and 48 sequences cross later, by up to four tiles, at 512 values in Q8_0 as early.)
    static constexpr int SHORT = Q8 ? (D == 64 ? 5 : D == 128 ? 3 : 2) : (D == 64 ? 8 : 5);
    static constexpr int NST = Q8 && D <= 128 ? 3 : 2;         // stages of a warp
    static constexpr bool QREG = D <= 128;               // q fragments in registers (else shared memory)
    static constexpr int QS = QREG ? 0 : D / 16 * NT * 256;   // q fragments, [k step][head tile][lane] of 8 bytes
    static constexpr int MERGE = HR * DV * 4;            // a warp's O at the end of a share
    static constexpr int RING = NST * STAGE > MERGE ? NST * STAGE : MERGE;
    static constexpr int SMEM = W * RING + QS + W * HR * 8 + 64 + 64;
    static constexpr int FIT = 224 * 1024 / SMEM;
    static constexpr int CTAS = FIT < 1 ? 1 : (D == 64 ? (FIT < 4 ? FIT : 4) : (D == 128 ? (FIT < 3 ? FIT : 3) : 1));
    static constexpr int UP = FMT == 1 ? 0 : 15;         // fp16 weights: the largest is 2^15 (weight_ref)
    static_assert(STAGE % 128 == 0, "stage alignment");
};

// 16-byte chunk of a staged row, permuted so that the fragment loads of a warp meet no bank twice.
template <int D, bool Q8, bool V> __device__ __forceinline__ int swz(int row, int chunk) {
    if constexpr (!Q8) return chunk ^ (row & 7);                     // ldmatrix: 8 rows, one chunk
    else if constexpr (V) return D >= 128 ? chunk ^ (((row >> 1) & 3) << 1) : chunk ^ (((row >> 2) & 1) << 1);
    else return D >= 128 ? chunk ^ ((row & 3) << 1) : chunk ^ (((row >> 1) & 1) << 1);
}

// Four biased bytes (q + 128) -> two pairs of exact 16-bit values.
template <bool BF16> __device__ __forceinline__ void bytes_to_pairs(uint32_t u, uint32_t &lo, uint32_t &hi) {
    if constexpr (!BF16) {
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));   // 1024 + 128
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
    } else {
        // bf16 holds 8 significant bits: 0x4300 is 128, whose low 7 mantissa bits are the integer
        // steps; bytes >= 128 (q >= 0) go through fp32 instead: exact for |q| <= 127.
        const float f0 = (float)((int)(u & 0xff) - 128), f1 = (float)((int)((u >> 8) & 0xff) - 128);
        const float f2 = (float)((int)((u >> 16) & 0xff) - 128), f3 = (float)((int)(u >> 24) - 128);
        lo = pack16<true>(f0, f1);
        hi = pack16<true>(f2, f3);
    }
}

// N 32-bit words of shared memory, N * 4 bytes aligned (at most 16).
template <int N> __device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t *p) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + 4 * i);
            w[i] = v.x;
            w[i + 1] = v.y;
            w[i + 2] = v.z;
            w[i + 3] = v.w;
        }
    }
}

// 8 x 8 16-bit matrix, two elements of row lane / 4 a thread, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, int FMT, int NT>
__global__ void __launch_bounds__(128, Dec<D, FMT, NT>::CTAS) k_attn_decode(const AttnDecodeParams p) {
    using C = Dec<D, FMT, NT>;
    constexpr bool BF16 = C::BF16, Q8 = C::Q8;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *qs = smem + C::W * C::RING;
    float2 *ml = reinterpret_cast<float2 *>(qs + C::QS);        // [warp][HR]
    int *sh = reinterpret_cast<int *>(ml + C::W * C::HR);          // small shared words
    float *sink = reinterpret_cast<float *>(sh + 16);               // the unit's heads' sinks, in log2 units
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    const int half = warp % C::NDH, slice = warp / C::NDH;
    uint8_t *ring = smem + warp * C::RING;
    const uint32_t ring_s = smem_addr(ring);
    grid_dep_wait();

    // ---- the line of tiles: this CTA's share, and the sequence it starts in
    const uint32_t units_per_seq = p.c.n_kv * p.mtiles;
    int64_t total, t0, t1;
    uint32_t s, shares;
    int64_t s_base;                                              // first tile of sequence s on the line
    bool by_unit;
    // a unit's length on the line
    auto on_line = [&](const Seq &q) { return by_unit ? min(q.tiles, 1) : (q.tiles ? q.tiles + HEAD : 0); };
    auto share_of = [&](int64_t n) {
        total = n;
        shares = n < (int64_t)gridDim.x ? (uint32_t)n : gridDim.x;   // every share has a tile
        t0 = t1 = 0;
        if (blockIdx.x >= shares) return;
        t0 = n * blockIdx.x / shares;
        t1 = n * (blockIdx.x + 1) / shares;
    };
    if (p.n_seq <= 32) {                                         // every warp for itself: no barriers
        const int n = lane < (int)p.n_seq ? seq_of(C::TT, 16, p, lane, blockIdx.x == 0 && warp == 0).tiles : 0;
        by_unit = __all_sync(0xffffffffu, n <= C::SHORT);
        const int64_t mine = (int64_t)(by_unit ? min(n, 1) : (n ? n + HEAD : 0)) * units_per_seq;
        int64_t sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        share_of(__shfl_sync(0xffffffffu, sum, 31));
        const uint32_t hit = __ballot_sync(0xffffffffu, t0 < t1 && sum - mine <= t0 && t0 < sum);
        s = hit ? (uint32_t)__ffs((int)hit) - 1 : 0;
        s_base = __shfl_sync(0xffffffffu, sum - mine, (int)s);
    } else {
        int64_t *scan = reinterpret_cast<int64_t *>(smem);       // before the ring is used
        const uint32_t per = (p.n_seq + 127) / 128, a = min(p.n_seq, tid * per), b = min(p.n_seq, a + per);
        int64_t mine = 0;
        int seen = 0, most = 0;                                  // sequences with tiles, the most tiles
#pragma unroll 8
        for (uint32_t i = a; i < b; ++i) {
            const int n = seq_of(C::TT, 16, p, i, blockIdx.x == 0).tiles;
            mine += n;
            seen += n > 0;
            most = max(most, n);
        }
        by_unit = !__syncthreads_or(most > C::SHORT);
        mine = by_unit ? seen : mine + (int64_t)HEAD * seen;
        mine *= units_per_seq;
        int64_t sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (lane == 31) scan[warp] = sum;
        __syncthreads();
        int64_t before = sum - mine;
        total = 0;
        for (int w = 0; w < 4; ++w) {
            if (w < warp) before += scan[w];
            total += scan[w];
        }
        share_of(total);
        // one thread's range holds t0 (when the share is not empty)
        if (t0 < t1 && before <= t0 && t0 < before + mine) {
            uint32_t i = a;
            for (;; ++i) {
                const int64_t n = (int64_t)on_line(seq_of(C::TT, 16, p, i, false)) * units_per_seq;
                if (t0 < before + n) break;
                before += n;
            }
            scan[8] = i;
            scan[9] = before;
        }
        __syncthreads();
        s = (uint32_t)scan[8];
        s_base = scan[9];
        __syncthreads();
    }

    // ---- sequences with nothing visible: zeros, 128 chunks of 8 values a CTA, those without a share first
    {
        const uint32_t items = p.n_heads * (D / 8), parts = (items + 127) / 128;
        const uint32_t from = (blockIdx.x + gridDim.x - shares) % gridDim.x;
        for (uint64_t w = from; w < (uint64_t)p.n_seq * parts; w += gridDim.x) {
            const uint32_t e = (uint32_t)(w / parts), i = (uint32_t)(w % parts) * 128 + tid;
            if (seq_of(C::TT, 16, p, e, false).tiles) continue;
            const bool act = i < items;
            const uint32_t head = act ? i / (D / 8) : 0;
            float o[8] = {};
            finish8(p, e, head, i % (D / 8) * 8, sink_of(p, head, act), -INFINITY, 0.0f, o, act);
        }
    }

    bool first = true;
    for (int64_t tile = t0; tile < t1; first = false) {
        Seq q = seq_of(C::TT, 16, p, s, false);
        while (tile >= s_base + (int64_t)on_line(q) * units_per_seq) {
            s_base += (int64_t)on_line(q) * units_per_seq;
            q = seq_of(C::TT, 16, p, ++s, false);
        }
        const int len = on_line(q);
        const uint32_t unit = (uint32_t)((tile - s_base) / len);
        const int64_t u0 = s_base + (int64_t)unit * len, u1 = u0 + len;   // the unit on the line
        const int ta = by_unit ? 0 : max((int)(tile - u0) - HEAD, 0);
        const int tb = by_unit ? q.tiles : (int)min((int64_t)len, t1 - u0) - HEAD;
        if (tb <= 0) break;                                      // the share ends before the unit's first tile
        const uint32_t kvh = unit / p.mtiles, mt = unit % p.mtiles;
        const uint32_t head0 = kvh * p.group + mt * C::HR;
        const int rows = (int)min((uint32_t)C::HR, p.group - mt * C::HR);

        if (p.sinks && tid < rows) sink[tid] = p.sinks[head0 + tid] * 1.4426950408889634f;   // read after the next barrier

        // ---- q fragments
        const uint16_t *qrow = static_cast<const uint16_t *>(p.q) + (uint64_t)s * p.q_stride + (uint64_t)head0 * D;
        // K step ks covers 16 values of head 8 t + g: a thread holds values k0, k0 + 1 and k1, k1 + 1, in the usual
        // order, or, for Q8_0, four in a row out of the eight that one thread reads from each block.
        auto qfrag = [&](int ks, int t, uint32_t (&f)[2]) {
            const int k0 = Q8 ? ks / 2 * 32 + 8 * c + ks % 2 * 4 : ks * 16 + 2 * c, k1 = Q8 ? k0 + 2 : k0 + 8;
            const uint16_t *r = qrow + (8 * t + g) * D;
            f[0] = 8 * t + g < rows ? *reinterpret_cast<const uint32_t *>(r + k0) : 0u;
            f[1] = 8 * t + g < rows ? *reinterpret_cast<const uint32_t *>(r + k1) : 0u;
        };
        uint32_t qr[C::QREG ? D / 16 : 1][NT][2];
        if constexpr (C::QREG) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int t = 0; t < NT; ++t) qfrag(ks, t, qr[ks][t]);
        } else {
#pragma unroll 8
            for (int i = warp; i < D / 16 * NT; i += C::W) {     // eight fragments' loads in flight
                uint32_t f[2];
                qfrag(i / NT, i % NT, f);
                reinterpret_cast<uint2 *>(qs)[i * 32 + lane] = make_uint2(f[0], f[1]);
            }
            __syncthreads();
        }
        auto q_of = [&](int ks, int t, uint32_t &b0, uint32_t &b1) {
            if constexpr (C::QREG) {
                b0 = qr[ks][t][0];
                b1 = qr[ks][t][1];
            } else {
                const uint2 f = reinterpret_cast<const uint2 *>(qs)[(ks * NT + t) * 32 + lane];
                b0 = f.x;
                b1 = f.y;
            }
        };

        // ---- staging: slice i of this warp covers positions pos0 + i * TT ..
        const int pos0 = q.start + ta * C::TT + slice * C::ST, n_it = tb - ta;
        const int32_t *pages = p.table + (uint64_t)s * p.table_stride;
        int pg_base = -1, pg = -1;                               // page ids of 32 sixteen-position pieces
        uint32_t dead_of = 0;                                    // two bits a stage: pieces without a page
        auto stage = [&](int it) {
            if (it < n_it) {
                const uint32_t st = ring_s + (it % C::NST) * C::STAGE;
                const int p0 = pos0 + it * C::TT;
                // page ids: lane j looks up piece j of the next 32 (ST / 16 pieces a slice)
                constexpr int NP = C::ST / 16;
                const int w0 = it * NP / 32 * 32;
                if (w0 != pg_base) {
                    pg_base = w0;
                    const int piece = w0 + lane, at = pos0 + piece / NP * C::TT + piece % NP * 16;
                    pg = -1;
                    if (piece < n_it * NP && at < q.hi) {
                        pg = pages[at >> p.c.page_shift];
                        if (pg < 0 || (uint32_t)pg >= p.c.n_pages) {
                            raise_error(p.err, DEV_ERANGE);
                            pg = -1;
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    const int id = __shfl_sync(0xffffffffu, pg, (it * NP + j) & 31);
                    const int bit = it % C::NST * 2 + j;
                    dead_of = (dead_of & ~(1u << bit)) | (id < 0 ? 1u << bit : 0u);
                    const int a = p0 + 16 * j;                   // 16 positions of one page
                    const uint64_t page = (uint64_t)max(id, 0) * p.c.page_stride + (uint64_t)kvh * p.c.tile_bytes;
                    const uint32_t in = (uint32_t)a & ((1u << p.c.page_shift) - 1u);
                    constexpr int ROW = D * (Q8 ? 1 : 2), CH = ROW / 16, VCH = C::DV * (Q8 ? 1 : 2) / 16;
                    const uint8_t *k = p.c.k + page + (uint64_t)in * ROW;
                    const uint8_t *v = p.c.v + page + (uint64_t)in * ROW + half * VCH * 16;
#pragma unroll
                    for (int e = 0; e < 16 * CH / 32; ++e) {
                        const int i = e * 32 + lane, r = i / CH, ch = i % CH;
                        const bool ok = id >= 0 && a + r >= q.lo && a + r < q.hi;
                        cp_async16(st + (16 * j + r) * ROW + swz<D, Q8, false>(16 * j + r, ch) * 16,
                                   ok ? k + r * ROW + ch * 16 : p.c.k, ok);
                    }
#pragma unroll
                    for (int e = 0; e < 16 * VCH / 32; ++e) {
                        const int i = e * 32 + lane, r = i / VCH, ch = i % VCH;
                        const bool ok = id >= 0 && a + r >= q.lo && a + r < q.hi;
                        cp_async16(st + C::KB + (16 * j + r) * (VCH * 16) + swz<C::DV, Q8, true>(16 * j + r, ch) * 16,
                                   ok ? v + r * ROW + ch * 16 : p.c.v, ok);
                    }
                    if constexpr (Q8) {                           // scales: not masked here, see below
                        constexpr int SR = D / 32 * 2, SV = C::DV / 32 * 2;   // bytes a position
                        const uint64_t so = page + ((uint64_t)D << p.c.page_shift) + (uint64_t)in * SR;
                        const bool ok = id >= 0 && a < q.hi;
#pragma unroll
                        for (int e = 0; e < (16 * SR + 511) / 512; ++e) {
                            const int i = e * 32 + lane;
                            if (i < SR) cp_async16(st + C::KB + C::VB + j * 16 * SR + i * 16, ok ? p.c.k + so + i * 16 : p.c.k, ok);
                        }
#pragma unroll
                        for (int e = 0; e < (16 * SV + 511) / 512; ++e) {
                            const int i = e * 32 + lane;
                            if (i < SV) {
                                // 16-byte piece i of this half's scales: whole rows back to back, or (two
                                // halves) the half of row i
                                const uint64_t o = C::NDH == 1 ? (uint64_t)i * 16 : (uint64_t)(i * 16 / SV) * SR + half * SV + i * 16 % SV;
                                cp_async16(st + C::KB + C::VB + C::KSB + j * 16 * SV + i * 16, ok ? p.c.v + so + o : p.c.v, ok);
                            }
                        }
                    }
                }
            }
            cp_async_commit();
        };

        // O, transposed: tile dt, head tile t: rows (dims) g and g + 8, columns (heads) 2c and 2c + 1
        float o[C::DV / 16][NT][4];
#pragma unroll
        for (int i = 0; i < C::DV / 16; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) o[i][t][0] = o[i][t][1] = o[i][t][2] = o[i][t][3] = 0.0f;
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < C::NST - 1; ++i) stage(i);

        for (int it = 0; it < n_it; ++it) {
            stage(it + C::NST - 1);
            cp_async_wait<C::NST - 1>();
            __syncwarp();
            const uint8_t *st = ring + (it % C::NST) * C::STAGE;
            const uint32_t st_s = ring_s + (it % C::NST) * C::STAGE;
            const int p0 = pos0 + it * C::TT;
            if (p0 < q.hi) {                                     // the last tile may end before this slice
                constexpr int MT = C::ST / 16;                   // tiles of 16 positions: rows g and g + 8
                float z[MT][NT][4];
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int t = 0; t < NT; ++t) z[i][t][0] = z[i][t][1] = z[i][t][2] = z[i][t][3] = 0.0f;
                // ---- scores
                if constexpr (!Q8) {
                    const int r = ((lane >> 3) & 1) * 8 + (lane & 7), hc = lane >> 4;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        uint32_t a[4];
                        ldsm4(a, st_s + r * (D * 2) + swz<D, Q8, false>(r, ks * 2 + hc) * 16);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            uint32_t b0, b1;
                            q_of(ks, t, b0, b1);
                            mma16<BF16>(z[0][t], a, b0, b1);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const int ra = 16 * i + g, rb = ra + 8;
                        uint32_t da[D / 64], db[D / 64];         // K scales of the thread's two positions
                        load_words<D / 64>(da, st + C::KB + C::VB + ra * (D / 16));
                        load_words<D / 64>(db, st + C::KB + C::VB + rb * (D / 16));
#pragma unroll
                        for (int b = 0; b < D / 32; ++b) {
                            const uint2 wa = *reinterpret_cast<const uint2 *>(st + ra * D + swz<D, true, false>(ra, 2 * b) * 16 + 8 * c);
                            const uint2 wb = *reinterpret_cast<const uint2 *>(st + rb * D + swz<D, true, false>(rb, 2 * b) * 16 + 8 * c);
                            uint32_t a0[4], a1[4];
                            bytes_to_pairs<BF16>(wa.x ^ 0x80808080u, a0[0], a0[2]);
                            bytes_to_pairs<BF16>(wb.x ^ 0x80808080u, a0[1], a0[3]);
                            bytes_to_pairs<BF16>(wa.y ^ 0x80808080u, a1[0], a1[2]);
                            bytes_to_pairs<BF16>(wb.y ^ 0x80808080u, a1[1], a1[3]);
                            const float sa = half_bits_to_float((uint16_t)(da[b / 2] >> (b % 2 * 16)));
                            const float sb = half_bits_to_float((uint16_t)(db[b / 2] >> (b % 2 * 16)));
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                uint32_t b0, b1;
                                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                q_of(2 * b, t, b0, b1);
                                mma16<BF16>(acc, a0, b0, b1);
                                q_of(2 * b + 1, t, b0, b1);
                                mma16<BF16>(acc, a1, b0, b1);
                                z[i][t][0] += acc[0] * sa;
                                z[i][t][1] += acc[1] * sa;
                                z[i][t][2] += acc[2] * sb;
                                z[i][t][3] += acc[3] * sb;
                            }
                        }
                    }
                }
                // ---- mask, running maximum
                const bool edge = p0 < q.lo || p0 + C::ST > q.hi;
                const uint32_t dead = (dead_of >> (it % C::NST * 2)) & (MT == 2 ? 3u : 1u);   // bit j: piece j
                float e_max = 0.0f;                              // Q8_0: |V scales| < 2^e_max
                const uint8_t *vs_s = st + C::KB + C::VB + C::KSB;
                if constexpr (Q8) {
                    const int at = p0 + lane;                    // one position a lane
                    uint32_t big = 0;
                    if (at >= q.lo && at < q.hi && !((dead >> (lane / 16)) & 1)) {
                        uint32_t w[C::DV / 64];
                        load_words<C::DV / 64>(w, vs_s + lane * (C::DV / 16));
#pragma unroll
                        for (int i = 0; i < C::DV / 64; ++i) big = max(big, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
                    }
                    big = __reduce_max_sync(0xffffffffu, big);
                    e_max = (float)((int)(big >> 10) - 14);
                }
                uint32_t seen = ~0u;                             // bit 2 i + h: position 16 i + g + 8 h
                if (edge || dead) {
                    seen = 0;
#pragma unroll
                    for (int i = 0; i < 2 * MT; ++i) {
                        const int at = p0 + 8 * i + g;
                        seen |= (uint32_t)(at >= q.lo && at < q.hi && !((dead >> (i / 2)) & 1)) << i;
                    }
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (!(seen & (1u << (2 * i + (e >> 1))))) z[i][t][e] = -INFINITY;
                }
                float mx[NT][2];
                bool grow = false;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    mx[t][0] = mx[t][1] = -INFINITY;
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            mx[t][e & 1] = fmaxf(mx[t][e & 1], z[i][t][e]);
                        }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) mx[t][h] = fmaxf(mx[t][h], __shfl_xor_sync(0xffffffffu, mx[t][h], x));
                        mx[t][h] = mx[t][h] * p.scale_log2 + e_max;
                        grow |= mx[t][h] > m[t][h];
                    }
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float mn = fmaxf(m[t][h], mx[t][h]);
                            const float f = m[t][h] == -INFINITY ? 0.0f : ex2(weight_ref<C::UP>(m[t][h]) - weight_ref<C::UP>(mn));
                            m[t][h] = mn;
                            l[t][h] *= f;
#pragma unroll
                            for (int i = 0; i < C::DV / 16; ++i) {
                                o[i][t][h] *= f;
                                o[i][t][2 + h] *= f;
                            }
                        }
                }
                // ---- weights
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float s = m[t][h] == -INFINITY ? 0.0f : -weight_ref<C::UP>(m[t][h]);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            z[i][t][h] = ex2(__fmaf_rn(z[i][t][h], p.scale_log2, s));
                            z[i][t][2 + h] = ex2(__fmaf_rn(z[i][t][2 + h], p.scale_log2, s));
                            l[t][h] += z[i][t][h] + z[i][t][2 + h];
                        }
                    }
                // ---- O^T += V^T P^T
                if constexpr (!Q8) {
                    uint32_t b[NT][2];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        b[t][0] = transpose8(pack16<BF16>(z[0][t][0], z[0][t][1]));
                        b[t][1] = transpose8(pack16<BF16>(z[0][t][2], z[0][t][3]));
                    }
                    const int r = (lane >> 4) * 8 + (lane & 7), hc = (lane >> 3) & 1;
#pragma unroll
                    for (int n = 0; n < C::DV / 16; ++n) {
                        uint32_t a[4];
                        ldsm4t(a, st_s + C::KB + r * (C::DV * 2) + swz<C::DV, Q8, true>(r, n * 2 + hc) * 16);
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma16<BF16>(o[n][t], a, b[t][0], b[t][1]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        // the weights carry the V scale of their position and block; nothing beside a masked
                        // position is used, whatever it holds
                        const int ra = 16 * i + g;
                        uint32_t da[C::DV / 64], db[C::DV / 64];
                        load_words<C::DV / 64>(da, vs_s + ra * (C::DV / 16));
                        load_words<C::DV / 64>(db, vs_s + (ra + 8) * (C::DV / 16));
                        const uint32_t ka = seen & (1u << (2 * i)) ? 0xffffffffu : 0u, kb = seen & (2u << (2 * i)) ? 0xffffffffu : 0u;
                        const int r0 = 16 * i + 2 * c;
#pragma unroll
                        for (int b = 0; b < C::DV / 32; ++b) {
                            const float sa = half_bits_to_float((uint16_t)((da[b / 2] & ka) >> (b % 2 * 16)));
                            const float sb = half_bits_to_float((uint16_t)((db[b / 2] & kb) >> (b % 2 * 16)));
                            // four dims (4g ..) of four positions: pairs along the positions
                            auto word = [&](int r) {
                                return *reinterpret_cast<const uint32_t *>(st + C::KB + r * C::DV +
                                                                           swz<C::DV, true, true>(r, 2 * b) * 16 + 4 * g) ^ 0x80808080u;
                            };
                            const uint32_t w0 = word(r0), w1 = word(r0 + 1), w8 = word(r0 + 8), w9 = word(r0 + 9);
                            uint32_t a0[4], a1[4];               // dims 4g, 4g + 1 and 4g + 2, 4g + 3 of the block
                            bytes_to_pairs<false>(__byte_perm(w0, w1, 0x5140), a0[0], a0[1]);
                            bytes_to_pairs<false>(__byte_perm(w0, w1, 0x7362), a1[0], a1[1]);
                            bytes_to_pairs<false>(__byte_perm(w8, w9, 0x5140), a0[2], a0[3]);
                            bytes_to_pairs<false>(__byte_perm(w8, w9, 0x7362), a1[2], a1[3]);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                const uint32_t b0 = transpose8(pack16<false>(z[i][t][0] * sa, z[i][t][1] * sa));
                                const uint32_t b1 = transpose8(pack16<false>(z[i][t][2] * sb, z[i][t][3] * sb));
                                mma16<false>(o[2 * b][t], a0, b0, b1);
                                mma16<false>(o[2 * b + 1][t], a1, b0, b1);
                            }
                        }
                    }
                }
            }
            __syncwarp();   // the stage is free for the copies of the next iteration
        }
        cp_async_wait<0>();

        // ---- the CTA's share of the unit: four warps' pieces joined
        float *mo = reinterpret_cast<float *>(ring);             // [HR][DV]
        __syncwarp();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[t][h] += __shfl_xor_sync(0xffffffffu, l[t][h], x);
                if (g == 0) ml[warp * C::HR + 8 * t + 2 * c + h] = make_float2(weight_ref<C::UP>(m[t][h]), l[t][h]);
#pragma unroll
                for (int i = 0; i < C::DV / 16; ++i) {
                    // Q8_0 tiles hold dims 4 g + 0, 1 and 4 g + 2, 3 of a block
                    float *dst = mo + (8 * t + 2 * c + h) * C::DV;
                    dst[Q8 ? i / 2 * 32 + 4 * g + i % 2 * 2 : 16 * i + g] = o[i][t][h];
                    dst[Q8 ? i / 2 * 32 + 4 * g + i % 2 * 2 + 1 : 16 * i + g + 8] = o[i][t][2 + h];
                }
            }
        __syncthreads();
        const bool whole = ta == 0 && tb == q.tiles;
        const uint64_t slot = 2 * (uint64_t)blockIdx.x + (first ? 0 : 1);
        const int items = rows * (D / 8);
        for (int i = tid; i < (items + 31) / 32 * 32; i += 128) {
            const bool act = i < items;
            const int row = act ? i / (D / 8) : 0, d0 = i % (D / 8) * 8, h = d0 / C::DV;
            float mt = -INFINITY, lt = 0.0f, y[8] = {};
#pragma unroll
            for (int w = 0; w < C::SL; ++w) mt = fmaxf(mt, ml[(w * C::NDH + h) * C::HR + row].x);
#pragma unroll
            for (int w = 0; w < C::SL; ++w) {
                const float2 x = ml[(w * C::NDH + h) * C::HR + row];
                const float f = x.x == -INFINITY ? 0.0f : ex2(x.x - mt);
                lt += x.y * f;
                const float *src = reinterpret_cast<const float *>(smem + (w * C::NDH + h) * C::RING) + row * C::DV + d0 % C::DV;
                float v[8];
                load8s(v, src);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] += v[e] * f;
            }
            if (whole) {
                finish8(p, s, head0 + row, d0, sink[row], mt, lt, y, act);
            } else if (act) {
                float4 *dst = reinterpret_cast<float4 *>(p.part + (slot * 16 + row) * D + d0);
                dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                dst[1] = make_float4(y[4], y[5], y[6], y[7]);
                // two halves of a head may carry different maxima (their V scales differ): one pair each
                if (d0 % C::DV == 0) p.part_ml[(slot * 16 + row) * 2 + h] = make_float2(mt, lt);
            }
        }
        if (!whole) {
            // pieces of the unit: CTAs c0 .. c1 of the line
            auto cta_of = [&](int64_t x) {                       // the CTA whose share holds tile x
                int64_t k = x * shares / total;
                while (total * (k + 1) / shares <= x) ++k;
                while (total * k / shares > x) --k;
                return k;
            };
            const int64_t c0 = cta_of(u0 + HEAD), c1 = cta_of(u1 - 1);
            const int n_part = (int)(c1 - c0) + 1;
            // the first piece is its CTA's second share when that CTA began with another unit
            const uint64_t first_slot = 2 * (uint64_t)c0 + (total * c0 / shares >= u0 ? 0 : 1);
            auto slot_of = [&](int k) { return k == 0 ? first_slot : 2 * (uint64_t)(c0 + k); };
            // Up to AT_ONCE pieces are joined by the last CTA to arrive.  Of more, each GROUP in a row are joined by the
            // last of them, in the place of the first, and the groups by the last of those.
            const int k_own = (int)(blockIdx.x - c0), k_first = n_part > AT_ONCE ? k_own / GROUP * GROUP : 0;
            const int n_own = min(GROUP, n_part - k_first);
            // whether this CTA is the last of n to arrive; the counter is then zero again
            auto last_of = [&](int *counter, int n) {
                __syncthreads();                                 // the whole CTA's piece before its arrival
                if (tid == 0) {
                    __threadfence();
                    sh[0] = atomicAdd(counter, 1) == n - 1;
                    if (sh[0]) *counter = 0;
                    __threadfence();
                }
                __syncthreads();
                return sh[0] != 0;
            };
            int *const unit_counter = p.counters + (uint64_t)s * units_per_seq + unit;
            int *const group_counter = p.counters + (uint64_t)p.n_seq * units_per_seq + slot_of(k_first);
            // pieces k0, k0 + step, .. (n of them): the result, or one piece in the place of the first
            auto join = [&](int k0, int step, int n, const float2 *from, bool result) {
                for (int i = tid; i < (items + 31) / 32 * 32; i += 128) {
                    const bool act = i < items;
                    const int row = act ? i / (D / 8) : 0, d0 = i % (D / 8) * 8, h = d0 / C::DV;
                    float mj, lj, y[8];
                    join8(n, [&](int k) { return p.part + (slot_of(k0 + k * step) * 16 + row) * D + d0; },
                          [&](int k) { return from + (slot_of(k0 + k * step) * 16 + row) * 2 + h; }, mj, lj, y);
                    if (result) {
                        finish8(p, s, head0 + row, d0, sink[row], mj, lj, y, act);
                    } else if (act) {
                        const uint64_t to = slot_of(k0) * 16 + row;
                        float4 *dst = reinterpret_cast<float4 *>(p.part + to * D + d0);
                        dst[0] = make_float4(y[0], y[1], y[2], y[3]);
                        dst[1] = make_float4(y[4], y[5], y[6], y[7]);
                        // beside the pieces' own, which other threads still read
                        if (d0 % C::DV == 0) p.group_ml[to * 2 + h] = make_float2(mj, lj);
                    }
                }
            };
            if (n_part <= AT_ONCE) {
                if (last_of(unit_counter, n_part)) join(0, 1, n_part, p.part_ml, true);
            } else if (last_of(group_counter, n_own)) {
                join(k_first, 1, n_own, p.part_ml, false);
                const int groups = (n_part + GROUP - 1) / GROUP;
                if (last_of(unit_counter, groups)) join(0, GROUP, groups, p.group_ml, true);
            }
        }
        __syncthreads();   // the rings, ml and sh are free again
        tile = min(u1, t1);
    }
}

template <int D, int FMT, int NT> cudaError_t launch_one(const AttnDecodeParams &p, int grid, cudaStream_t st) {
    static SmemAllowed allowed;
    const cudaError_t es = allow_smem(allowed, reinterpret_cast<const void *>(k_attn_decode<D, FMT, NT>), Dec<D, FMT, NT>::SMEM);
    if (es != cudaSuccess) return es;
    return launch_dependent(k_attn_decode<D, FMT, NT>, p, dim3((unsigned)grid), 128, Dec<D, FMT, NT>::SMEM, st);
}

template <int D, int NT> cudaError_t launch_dim(const AttnDecodeParams &p, int grid, cudaStream_t st) {
    const bool bf = p.q_type == Q8_TYPE_BF16;
    if (p.c.type == Q8_TYPE_Q8_0) return bf ? launch_one<D, 3, NT>(p, grid, st) : launch_one<D, 2, NT>(p, grid, st);
    return bf ? launch_one<D, 1, NT>(p, grid, st) : launch_one<D, 0, NT>(p, grid, st);
}

template <int D> cudaError_t launch_heads(const AttnDecodeParams &p, int grid, cudaStream_t st) {
    return attn_decode_heads(p.group) == 8 ? launch_dim<D, 1>(p, grid, st) : launch_dim<D, 2>(p, grid, st);
}

template <int D> int grid_of(uint32_t group, int cache_type, int num_sms) {
    const bool q8 = cache_type == Q8_TYPE_Q8_0;
    if (attn_decode_heads(group) == 8) return num_sms * (q8 ? Dec<D, 2, 1>::CTAS : Dec<D, 0, 1>::CTAS);
    return num_sms * (q8 ? Dec<D, 2, 2>::CTAS : Dec<D, 0, 2>::CTAS);
}

}  // namespace

int attn_decode_grid(uint32_t dim, uint32_t group, int cache_type, int num_sms) {
    switch (dim) {
        case 64: return grid_of<64>(group, cache_type, num_sms);
        case 128: return grid_of<128>(group, cache_type, num_sms);
        case 256: return grid_of<256>(group, cache_type, num_sms);
        case 512: return grid_of<512>(group, cache_type, num_sms);
        default: return 0;
    }
}

cudaError_t launch_attn_decode(const AttnDecodeParams &p, int grid, cudaStream_t st) {
    switch (p.c.dim) {
        case 64: return launch_heads<64>(p, grid, st);
        case 128: return launch_heads<128>(p, grid, st);
        case 256: return launch_heads<256>(p, grid, st);
        case 512: return launch_heads<512>(p, grid, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace q8
