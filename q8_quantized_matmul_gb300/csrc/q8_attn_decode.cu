// q8_attn_decode.cu -- attention of one new token per sequence over a paged cache.
//
//   z_j = scale q.k_j,  out = sum_j 2^(z_j - m) v_j / (sum_j 2^(z_j - m) + 2^(sink - m))   (z in log2 units)
//
// One pass over the visible positions with a running maximum m, sum l and unnormalised output O
// (all fp32).  Every cached byte is read once, so HBM is the bound: 2 D values per position and
// key-value head against 4 D operations per query head.
//
// Split.  A unit is (sequence, key-value head, tile of 16 of its query heads): those heads share every
// K and V row and fill the 16 rows of an mma.sync tile (fewer heads leave rows idle; the tensor pipe
// has the room).  The units' positions, in tiles of TT, form one line that is cut into equal shares,
// one per CTA, so the lengths do not matter to the balance.  A CTA that covers a whole unit writes its
// result; otherwise it leaves (m, l, O) in scratch, and the last CTA of a unit to arrive (one counter
// per unit, set back to zero by it) joins the pieces in their order: the same bits on every run.
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
// products stay below 2^15 and the weights keep 29 binades above the smallest normal.
#include <algorithm>

#include "q8_attn.cuh"
#include "q8_kv.h"

namespace q8 {
namespace {

template <int D, int FMT> struct Dec {   // FMT 0: f16, 1: bf16, 2: Q8_0 with f16 q, 3: Q8_0 with bf16 q
    static constexpr bool Q8 = FMT >= 2, BF16 = FMT & 1;
    static constexpr int W = 4;                          // warps
    static constexpr int ST = Q8 ? 32 : 16;              // positions of a warp's slice
    static constexpr int DV = D > 256 ? 256 : D;         // V dimensions of a warp
    static constexpr int NDH = D / DV;                   // warps that share a slice
    static constexpr int SL = W / NDH;                   // slices in a tile
    static constexpr int TT = SL * ST;                   // positions of a tile
    static constexpr int KB = ST * D * (Q8 ? 1 : 2), VB = ST * DV * (Q8 ? 1 : 2);
    static constexpr int KSB = Q8 ? ST * (D / 32) * 2 : 0, VSB = Q8 ? ST * (DV / 32) * 2 : 0;
    static constexpr int STAGE = KB + VB + KSB + VSB;
    static constexpr int NST = D <= 128 ? 3 : 2;         // stages of a warp
    static constexpr bool QREG = D <= 128;               // q fragments in registers (else shared memory)
    static constexpr int QS = QREG ? 0 : D / 16 * 512;   // q fragments, [k step][lane] of 16 bytes
    static constexpr int MERGE = 16 * DV * 4;            // a warp's O at the end of a share
    static constexpr int RING = NST * STAGE > MERGE ? NST * STAGE : MERGE;
    static constexpr int SMEM = W * RING + QS + W * 16 * 8 + 64;
    static constexpr int CTAS = SMEM * 4 <= 220 * 1024 && D < 128 ? 4 : (SMEM * 2 <= 220 * 1024 && D <= 128 ? 2 : 1);
    static constexpr float BIAS = Q8 ? 15.0f : 0.0f;     // weights are 2^(z - M + BIAS)
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

struct Seq {
    int lo, hi;          // visible positions [lo, hi)
    int start;           // lo rounded down to 16: the first staged position
    int tiles;
};

template <class C> __device__ __forceinline__ Seq seq_of(const AttnDecodeParams &p, uint32_t s, bool raise) {
    const int64_t most = (int64_t)p.max_pages << p.c.page_shift;
    int64_t n = p.lens[s];
    if (n < 0 || n > most) {
        if (raise) raise_error(p.err, DEV_ERANGE);
        n = n < 0 ? 0 : most;
    }
    Seq q;
    q.hi = (int)n;
    q.lo = p.window && n > p.window ? (int)(n - p.window) : 0;
    q.start = q.lo & ~15;
    q.tiles = (q.hi - q.start + C::TT - 1) / C::TT;
    return q;
}

// Final values of one output chunk (8 dims of a head).
__device__ __forceinline__ void finish8(const AttnDecodeParams &p, uint32_t s, uint32_t head, int d0, float m, float l,
                                        float (&o)[8], bool active) {
    float lse;
    const float f = softmax_finish(m, l, p.sinks != nullptr, p.sinks && active ? p.sinks[head] * 1.4426950408889634f : 0.0f,
                                   lse);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = f == 0.0f ? 0.0f : o[e] * f;
    const uint64_t row = (uint64_t)s * p.n_heads + head;
    store_out8(p.out, p.out_type, row * p.c.dim + d0, o, active);
    if (active && p.lse && d0 == 0) p.lse[row] = lse;
}

template <int D, int FMT> __global__ void __launch_bounds__(128, Dec<D, FMT>::CTAS) k_attn_decode(const AttnDecodeParams p) {
    using C = Dec<D, FMT>;
    constexpr bool BF16 = C::BF16, Q8 = C::Q8;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *qs = smem + C::W * C::RING;
    float2 *ml = reinterpret_cast<float2 *>(qs + C::QS);        // [warp][16]
    int *sh = reinterpret_cast<int *>(ml + C::W * 16);          // small shared words
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
    {
        int64_t *scan = reinterpret_cast<int64_t *>(smem);       // before the ring is used
        const uint32_t per = (p.n_seq + 127) / 128, a = min(p.n_seq, tid * per), b = min(p.n_seq, a + per);
        int64_t mine = 0;
        for (uint32_t i = a; i < b; ++i) mine += seq_of<C>(p, i, blockIdx.x == 0).tiles;
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
        shares = total < (int64_t)gridDim.x ? (uint32_t)total : gridDim.x;   // every share has a tile
        if (blockIdx.x < shares) {
            t0 = total * blockIdx.x / shares;
            t1 = total * (blockIdx.x + 1) / shares;
        } else {
            t0 = t1 = 0;
        }
        // one thread's range holds t0 (when the share is not empty)
        if (t0 < t1 && before <= t0 && t0 < before + mine) {
            uint32_t i = a;
            for (;; ++i) {
                const int64_t n = (int64_t)seq_of<C>(p, i, false).tiles * units_per_seq;
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

    // ---- sequences with nothing visible: zeros
    for (uint32_t e = blockIdx.x; e < p.n_seq; e += gridDim.x) {
        if (seq_of<C>(p, e, false).tiles) continue;
        for (uint32_t i = tid; i < (p.n_heads * (D / 8) + 31) / 32 * 32; i += 128) {
            float o[8] = {};
            const bool act = i < p.n_heads * (D / 8);
            finish8(p, e, act ? i / (D / 8) : 0, i % (D / 8) * 8, -INFINITY, 0.0f, o, act);
        }
    }

    bool first = true;
    for (int64_t t = t0; t < t1; first = false) {
        Seq q = seq_of<C>(p, s, false);
        while (t >= s_base + (int64_t)q.tiles * units_per_seq) {
            s_base += (int64_t)q.tiles * units_per_seq;
            q = seq_of<C>(p, ++s, false);
        }
        const uint32_t unit = (uint32_t)((t - s_base) / q.tiles);
        const int64_t u0 = s_base + (int64_t)unit * q.tiles;     // the unit's tiles on the line
        const int ta = (int)(t - u0), tb = (int)min((int64_t)q.tiles, t1 - u0);
        const uint32_t kvh = unit / p.mtiles, mt = unit % p.mtiles;
        const uint32_t head0 = kvh * p.group + mt * 16;
        const int rows = (int)min(16u, p.group - mt * 16);
        const bool two = rows > 8;

        // ---- q fragments
        const uint16_t *qrow = static_cast<const uint16_t *>(p.q) + (uint64_t)s * p.q_stride + (uint64_t)head0 * D;
        // K step ks covers 16 values; in a thread's fragment a0, a1 (rows g, g + 8) hold values k0, k0 + 1
        // and a2, a3 values k1, k1 + 1: of 16 in the usual order, or, for Q8_0, four in a row out of the
        // eight that one thread reads from each block.
        auto qfrag = [&](int ks, uint32_t (&f)[4]) {
            const int k0 = Q8 ? ks / 2 * 32 + 8 * c + ks % 2 * 4 : ks * 16 + 2 * c, k1 = Q8 ? k0 + 2 : k0 + 8;
            const uint16_t *ra = qrow + g * D, *rb = ra + 8 * D;
            f[0] = g < rows ? *reinterpret_cast<const uint32_t *>(ra + k0) : 0u;
            f[1] = g + 8 < rows ? *reinterpret_cast<const uint32_t *>(rb + k0) : 0u;
            f[2] = g < rows ? *reinterpret_cast<const uint32_t *>(ra + k1) : 0u;
            f[3] = g + 8 < rows ? *reinterpret_cast<const uint32_t *>(rb + k1) : 0u;
        };
        uint32_t qr[C::QREG ? D / 16 : 1][4];
        if constexpr (C::QREG) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) qfrag(ks, qr[ks]);
        } else {
            for (int ks = warp; ks < D / 16; ks += C::W) {
                uint32_t f[4];
                qfrag(ks, f);
                reinterpret_cast<uint4 *>(qs)[ks * 32 + lane] = make_uint4(f[0], f[1], f[2], f[3]);
            }
            __syncthreads();
        }

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
                    const uint64_t tile = (uint64_t)max(id, 0) * p.c.page_stride + (uint64_t)kvh * p.c.tile_bytes;
                    const uint32_t in = (uint32_t)a & ((1u << p.c.page_shift) - 1u);
                    constexpr int ROW = D * (Q8 ? 1 : 2), CH = ROW / 16, VCH = C::DV * (Q8 ? 1 : 2) / 16;
                    const uint8_t *k = p.c.k + tile + (uint64_t)in * ROW;
                    const uint8_t *v = p.c.v + tile + (uint64_t)in * ROW + half * VCH * 16;
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
                        const uint64_t so = tile + ((uint64_t)D << p.c.page_shift) + (uint64_t)in * SR;
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

        float o[C::DV / 8][4];
#pragma unroll
        for (int i = 0; i < C::DV / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
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
                constexpr int NT = C::ST / 8;
                float z[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) z[n][0] = z[n][1] = z[n][2] = z[n][3] = 0.0f;
                // ---- scores
                if constexpr (!Q8) {
                    const int r = (lane >> 4) * 8 + (lane & 7), hc = (lane >> 3) & 1;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        uint32_t b[4];
                        ldsm4(b, st_s + r * (D * 2) + swz<D, Q8, false>(r, ks * 2 + hc) * 16);
                        if constexpr (C::QREG) {
                            mma16<BF16>(z[0], qr[ks], b[0], b[1]);
                            mma16<BF16>(z[1], qr[ks], b[2], b[3]);
                        } else {
                            const uint4 f = reinterpret_cast<const uint4 *>(qs)[ks * 32 + lane];
                            const uint32_t a[4] = {f.x, f.y, f.z, f.w};
                            mma16<BF16>(z[0], a, b[0], b[1]);
                            mma16<BF16>(z[1], a, b[2], b[3]);
                        }
                    }
                } else {
                    const uint16_t *ks_s = reinterpret_cast<const uint16_t *>(st + C::KB + C::VB);
#pragma unroll
                    for (int b = 0; b < D / 32; ++b) {
                        uint32_t a0[4], a1[4];
                        if constexpr (C::QREG) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                a0[i] = qr[2 * b][i];
                                a1[i] = qr[2 * b + 1][i];
                            }
                        } else {
                            const uint4 f0 = reinterpret_cast<const uint4 *>(qs)[2 * b * 32 + lane];
                            const uint4 f1 = reinterpret_cast<const uint4 *>(qs)[(2 * b + 1) * 32 + lane];
                            a0[0] = f0.x; a0[1] = f0.y; a0[2] = f0.z; a0[3] = f0.w;
                            a1[0] = f1.x; a1[1] = f1.y; a1[2] = f1.z; a1[3] = f1.w;
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const int r = 8 * n + g, ch = swz<D, true, false>(r, 2 * b);
                            const uint2 w = *reinterpret_cast<const uint2 *>(st + r * D + ch * 16 + 8 * c);
                            uint32_t b0, b1, b2, b3;
                            bytes_to_pairs<BF16>(w.x ^ 0x80808080u, b0, b1);
                            bytes_to_pairs<BF16>(w.y ^ 0x80808080u, b2, b3);
                            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma16<BF16>(acc, a0, b0, b1);
                            mma16<BF16>(acc, a1, b2, b3);
                            const float d0 = half_bits_to_float(ks_s[(8 * n + 2 * c) * (D / 32) + b]);
                            const float d1 = half_bits_to_float(ks_s[(8 * n + 2 * c + 1) * (D / 32) + b]);
                            z[n][0] += acc[0] * d0;
                            z[n][1] += acc[1] * d1;
                            z[n][2] += acc[2] * d0;
                            z[n][3] += acc[3] * d1;
                        }
                    }
                }
                // ---- mask, running maximum
                const bool edge = p0 < q.lo || p0 + C::ST > q.hi;
                const uint32_t dead = (dead_of >> (it % C::NST * 2)) & (C::ST / 16 == 2 ? 3u : 1u);   // bit j: piece j
                float e_max = 0.0f;                              // Q8_0: |V scales| < 2^e_max
                const uint16_t *vs_s = reinterpret_cast<const uint16_t *>(st + C::KB + C::VB + C::KSB);
                if constexpr (Q8) {
                    const int at = p0 + lane;                    // one position a lane
                    uint32_t big = 0;
                    if (at >= q.lo && at < q.hi && !((dead >> (lane / 16)) & 1))
#pragma unroll
                        for (int i = 0; i < C::DV / 32; ++i) big = max(big, (uint32_t)vs_s[lane * (C::DV / 32) + i] & 0x7fffu);
                    big = __reduce_max_sync(0xffffffffu, big);
                    e_max = (float)((int)(big >> 10) - 14);
                }
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v = z[n][i] * p.scale_log2;
                        if (edge || dead) {
                            const int at = p0 + 8 * n + 2 * c + (i & 1);
                            if (at < q.lo || at >= q.hi || ((dead >> (n / 2)) & 1)) v = -INFINITY;
                        }
                        z[n][i] = v;
                        mx[i >> 1] = fmaxf(mx[i >> 1], v);
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
                    mx[h] += e_max;
                }
                const bool grow = mx[0] > m[0] || mx[1] > m[1];
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float mn = fmaxf(m[h], mx[h]);
                        const float f = m[h] == -INFINITY ? 0.0f : ex2(m[h] - mn);
                        m[h] = mn;
                        l[h] *= f;
#pragma unroll
                        for (int i = 0; i < C::DV / 8; ++i) {
                            o[i][2 * h] *= f;
                            o[i][2 * h + 1] *= f;
                        }
                    }
                }
                // ---- weights
                const float s0 = m[0] == -INFINITY ? 0.0f : m[0] - C::BIAS, s1 = m[1] == -INFINITY ? 0.0f : m[1] - C::BIAS;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    z[n][0] = ex2(z[n][0] - s0);
                    z[n][1] = ex2(z[n][1] - s0);
                    l[0] += z[n][0] + z[n][1];
                    if (two) {
                        z[n][2] = ex2(z[n][2] - s1);
                        z[n][3] = ex2(z[n][3] - s1);
                        l[1] += z[n][2] + z[n][3];
                    } else {
                        z[n][2] = z[n][3] = 0.0f;
                    }
                }
                // ---- O += P V
                if constexpr (!Q8) {
                    const uint32_t a[4] = {pack16<BF16>(z[0][0], z[0][1]), pack16<BF16>(z[0][2], z[0][3]),
                                           pack16<BF16>(z[1][0], z[1][1]), pack16<BF16>(z[1][2], z[1][3])};
                    const int r = ((lane >> 3) & 1) * 8 + (lane & 7), hc = lane >> 4;
#pragma unroll
                    for (int n = 0; n < C::DV / 16; ++n) {
                        uint32_t b[4];
                        ldsm4t(b, st_s + C::KB + r * (C::DV * 2) + swz<C::DV, Q8, true>(r, n * 2 + hc) * 16);
                        mma16<BF16>(o[2 * n], a, b[0], b[1]);
                        mma16<BF16>(o[2 * n + 1], a, b[2], b[3]);
                    }
                } else {
                    // weights carry the V scale of their position and block; a masked weight is 0 whatever
                    // the scale beside it holds
                    auto w = [](float pz, uint16_t d) { return pz == 0.0f ? 0.0f : pz * half_bits_to_float(d); };
#pragma unroll
                    for (int kk = 0; kk < C::ST / 16; ++kk) {
#pragma unroll
                        for (int b = 0; b < C::DV / 32; ++b) {
                            const int r0 = 16 * kk + 2 * c;
                            const uint16_t d0 = vs_s[r0 * (C::DV / 32) + b], d1 = vs_s[(r0 + 1) * (C::DV / 32) + b];
                            const uint16_t d8 = vs_s[(r0 + 8) * (C::DV / 32) + b], d9 = vs_s[(r0 + 9) * (C::DV / 32) + b];
                            const float(&za)[4] = z[2 * kk];
                            const float(&zb)[4] = z[2 * kk + 1];
                            const uint32_t a[4] = {pack16<false>(w(za[0], d0), w(za[1], d1)),
                                                   pack16<false>(w(za[2], d0), w(za[3], d1)),
                                                   pack16<false>(w(zb[0], d8), w(zb[1], d9)),
                                                   pack16<false>(w(zb[2], d8), w(zb[3], d9))};
                            // four dims (4g ..) of four positions: pairs along the positions
                            auto word = [&](int r) {
                                const int ch = swz<C::DV, true, true>(r, 2 * b);
                                return *reinterpret_cast<const uint32_t *>(st + C::KB + r * C::DV + ch * 16 + 4 * g) ^ 0x80808080u;
                            };
                            const uint32_t w0 = word(r0), w1 = word(r0 + 1), w8 = word(r0 + 8), w9 = word(r0 + 9);
                            uint32_t x0, x1, x2, x3, y0, y1, y2, y3;
                            bytes_to_pairs<false>(__byte_perm(w0, w1, 0x5140), x0, x1);
                            bytes_to_pairs<false>(__byte_perm(w0, w1, 0x7362), x2, x3);
                            bytes_to_pairs<false>(__byte_perm(w8, w9, 0x5140), y0, y1);
                            bytes_to_pairs<false>(__byte_perm(w8, w9, 0x7362), y2, y3);
                            // column g of tile 4b + j is dim 32b + 4g + j
                            mma16<false>(o[4 * b], a, x0, y0);
                            mma16<false>(o[4 * b + 1], a, x1, y1);
                            mma16<false>(o[4 * b + 2], a, x2, y2);
                            mma16<false>(o[4 * b + 3], a, x3, y3);
                        }
                    }
                }
            }
            __syncwarp();   // the stage is free for the copies of the next iteration
        }
        cp_async_wait<0>();

        // ---- the CTA's share of the unit: four warps' pieces joined
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
        float *mo = reinterpret_cast<float *>(ring);             // [16][DV]
        __syncwarp();
#pragma unroll
        for (int i = 0; i < C::DV / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // accumulator columns 2c, 2c + 1 of tile i; Q8_0 tiles interleave their block's dims by four
                const int col = Q8 ? i / 4 * 32 + 4 * (2 * c + (e & 1)) + i % 4 : 8 * i + 2 * c + (e & 1);
                mo[(g + (e >> 1) * 8) * C::DV + col] = o[i][e];
            }
        if (c == 0) {
            ml[warp * 16 + g] = make_float2(m[0], l[0]);
            ml[warp * 16 + g + 8] = make_float2(m[1], l[1]);
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
            for (int w = 0; w < C::SL; ++w) mt = fmaxf(mt, ml[(w * C::NDH + h) * 16 + row].x);
#pragma unroll
            for (int w = 0; w < C::SL; ++w) {
                const float2 x = ml[(w * C::NDH + h) * 16 + row];
                const float f = x.x == -INFINITY ? 0.0f : ex2(x.x - mt);
                lt += x.y * f;
                const float *src = reinterpret_cast<const float *>(smem + (w * C::NDH + h) * C::RING) + row * C::DV + d0 % C::DV;
                float v[8];
                load8s(v, src);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] += v[e] * f;
            }
            if (whole) {
                finish8(p, s, head0 + row, d0, mt - C::BIAS, lt, y, act);
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
            const int64_t u1 = u0 + q.tiles;
            auto cta_of = [&](int64_t x) {                       // the CTA whose share holds tile x
                int64_t k = x * shares / total;
                while (total * (k + 1) / shares <= x) ++k;
                while (total * k / shares > x) --k;
                return k;
            };
            const int64_t c0 = cta_of(u0), c1 = cta_of(u1 - 1);
            __threadfence();
            __syncthreads();
            const uint64_t id = (uint64_t)s * units_per_seq + unit;
            if (tid == 0) sh[0] = atomicAdd(p.counters + id, 1) == (int)(c1 - c0);
            __syncthreads();
            if (sh[0]) {                                         // the last piece: join them in order
                __threadfence();
                const bool c0_first = total * c0 / shares == u0;   // the unit opens that share
                for (int i = tid; i < (items + 31) / 32 * 32; i += 128) {
                    const bool act = i < items;
                    const int row = act ? i / (D / 8) : 0, d0 = i % (D / 8) * 8, h = d0 / C::DV;
                    float mt = -INFINITY, lt = 0.0f, y[8] = {};
                    for (int64_t k = c0; k <= c1; ++k) {
                        const uint64_t sl = 2 * (uint64_t)k + (k == c0 && !c0_first ? 1 : 0);
                        const float2 x = __ldcg(&p.part_ml[(sl * 16 + row) * 2 + h]);
                        const float4 *src = reinterpret_cast<const float4 *>(p.part + (sl * 16 + row) * D + d0);
                        const float4 va = __ldcg(src), vb = __ldcg(src + 1);
                        const float mn = fmaxf(mt, x.x);
                        const float fo = mt == -INFINITY ? 0.0f : ex2(mt - mn), fn = x.x == -INFINITY ? 0.0f : ex2(x.x - mn);
                        mt = mn;
                        lt = lt * fo + x.y * fn;
                        const float v[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = y[e] * fo + v[e] * fn;
                    }
                    finish8(p, s, head0 + row, d0, mt - C::BIAS, lt, y, act);
                }
                if (tid == 0) p.counters[id] = 0;
            }
        }
        __syncthreads();   // the rings, ml and sh are free again
        t = u0 + tb;
    }
}

template <int D, int FMT> int grid_of(int num_sms) { return num_sms * Dec<D, FMT>::CTAS; }

template <int D, int FMT> cudaError_t launch_one(const AttnDecodeParams &p, int grid, cudaStream_t st) {
    static bool attr_done = false;
    if (!attr_done) {
        const cudaError_t e = cudaFuncSetAttribute(k_attn_decode<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   Dec<D, FMT>::SMEM);
        if (e != cudaSuccess) return e;
        attr_done = true;
    }
    return launch_dependent(k_attn_decode<D, FMT>, p, dim3((unsigned)grid), 128, Dec<D, FMT>::SMEM, st);
}

template <int D> cudaError_t launch_dim(const AttnDecodeParams &p, int grid, cudaStream_t st) {
    const bool bf = p.q_type == Q8_TYPE_BF16;
    if (p.c.type == Q8_TYPE_Q8_0) return bf ? launch_one<D, 3>(p, grid, st) : launch_one<D, 2>(p, grid, st);
    return bf ? launch_one<D, 1>(p, grid, st) : launch_one<D, 0>(p, grid, st);
}

template <int D> int grid_dim_of(int cache_type, int num_sms) {
    return cache_type == Q8_TYPE_Q8_0 ? grid_of<D, 2>(num_sms) : grid_of<D, 0>(num_sms);
}

}  // namespace

int attn_decode_grid(uint32_t dim, int cache_type, int num_sms) {
    switch (dim) {
        case 64: return grid_dim_of<64>(cache_type, num_sms);
        case 128: return grid_dim_of<128>(cache_type, num_sms);
        case 256: return grid_dim_of<256>(cache_type, num_sms);
        case 512: return grid_dim_of<512>(cache_type, num_sms);
        default: return 0;
    }
}

cudaError_t launch_attn_decode(const AttnDecodeParams &p, int grid, cudaStream_t st) {
    switch (p.c.dim) {
        case 64: return launch_dim<64>(p, grid, st);
        case 128: return launch_dim<128>(p, grid, st);
        case 256: return launch_dim<256>(p, grid, st);
        case 512: return launch_dim<512>(p, grid, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace q8
