// q8_attn_prompt.cuh -- what the prompt attention kernels share: which rows a CTA works on, which
// keys they see, and the handling of values that are not finite where some rows may not see them.
#pragma once

#include "q8_attn.cuh"
#include "q8_kv.h"

namespace q8 {

// Up to tile_tokens queries of one sequence (a row is a query token here, whatever heads are packed with it).
struct alignas(8) PromptTile {
    int q0, k0;          // first packed row of the sequence's queries / keys
    int row0, rows;      // first query of the tile within the sequence, and how many
    int lk, shift;       // keys; query i (of the sequence) sees keys up to i + shift

    // newest and oldest key that row r of the tile sees (none: last < first)
    __device__ __forceinline__ int last(int r) const { return row0 + r + shift; }
    __device__ __forceinline__ int first(int r, uint32_t window) const {
        const int64_t f = window ? (int64_t)last(r) - window + 1 : 0;
        return f > 0 ? (int)f : 0;
    }
    // Keys [key, key + n) that not every row of the tile sees.
    __device__ __forceinline__ bool masked(int key, int n, uint32_t window) const {
        return key + n - 1 > last(0) || key < first(rows - 1, window);
    }
};

__device__ __forceinline__ int prompt_bound(int32_t start, uint32_t n) { return (int)min((uint32_t)max(start, 0), n); }

// Tile `slot` of the packed sequences in tiles of BM queries, the newest rows of the last sequence
// first (their rows see the most keys, so the long tiles start first).  False: no such tile.
// Called by a whole CTA of THREADS; sh: THREADS / 32 + 5 ints of shared memory.  report: raise bad starts.
template <int THREADS>
__device__ __forceinline__ bool prompt_tile(const AttnPromptParams &p, int BM, uint32_t slot, bool report, PromptTile &w,
                                            int *sh) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int32_t *ks = p.k_start ? p.k_start : p.q_start;
    int tiles, qa, qe, ka, ke;
    auto sequence = [&](uint32_t i) {                // the i-th from the last
        tiles = qa = qe = ka = ke = 0;
        if (i >= p.n_seq) return;
        const uint32_t s = p.n_seq - 1 - i;
        const int4 raw = make_int4(p.q_start[s], p.q_start[s + 1], ks[s], ks[s + 1]);
        qa = prompt_bound(raw.x, p.n_q);
        qe = prompt_bound(raw.y, p.n_q);
        ka = prompt_bound(raw.z, p.n_k);
        ke = prompt_bound(raw.w, p.n_k);
        tiles = qe > qa ? (qe - qa + BM - 1) / BM : 0;
        if (report && (qe < qa || ke < ka || qa != raw.x || qe != raw.y || ka != raw.z || ke != raw.w))
            raise_error(p.err, DEV_ERANGE);
    };
    auto sum_to = [&](int sum) {                     // inclusive, over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        return sum;
    };
    auto claim = [&](int64_t at) {                   // this thread's sequence holds the tiles from `at` on
        if (tiles && slot >= at && slot < at + tiles) {
            sh[0] = (int)(at + tiles - 1 - slot);    // newest tile first
            int *b4 = sh + THREADS / 32 + 1;
            b4[0] = qa;
            b4[1] = qe - qa;
            b4[2] = ka;
            b4[3] = max(ke - ka, 0);
        }
    };
    if (p.n_seq <= 32) {                             // one warp, one barrier
        if (tid < 32) {
            if (lane == 0) sh[0] = -1;
            __syncwarp();
            sequence(lane);
            claim(sum_to(tiles) - tiles);
        }
        __syncthreads();
    } else {
        if (tid == 0) sh[0] = -1;
        __syncthreads();
        // sequences from the last one on, THREADS at a time
        int64_t before = 0;
        for (uint32_t b = 0; b < p.n_seq; b += THREADS) {
            sequence(b + tid);
            const int sum = sum_to(tiles);
            if (lane == 31) sh[1 + tid / 32] = sum;
            __syncthreads();
            int64_t at = before + sum - tiles;
            for (int k = 0; k < THREADS / 32; ++k) {
                if (k < tid / 32) at += sh[1 + k];
                before += sh[1 + k];
            }
            claim(at);
            __syncthreads();
            if (sh[0] >= 0) break;
        }
    }
    if (sh[0] < 0) return false;
    const int *b4 = sh + THREADS / 32 + 1;
    w.q0 = b4[0];
    w.k0 = b4[2];
    w.lk = b4[3];
    w.row0 = sh[0] * BM;
    w.rows = min(BM, b4[1] - w.row0);
    w.shift = w.lk - b4[1];
    return true;
}

// Sets 16-bit values that are not finite to zero.
template <bool BF16> __device__ __forceinline__ void prompt_scrub(uint4 &x) {
    constexpr uint32_t E = BF16 ? 0x7f80u : 0x7c00u;
    uint32_t *w = &x.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & E) == E) w[i] &= 0xffff0000u;
        if ((w[i] & (E << 16)) == E << 16) w[i] &= 0x0000ffffu;
    }
}

// The same for a tile of N / 16 16-byte words in shared memory, by 64 threads (t: 0 .. 63); *dirty = mark if there were
// any.  Eight words are loaded at once and looked at through one packed maximum: a word after the other took 1 us longer
// before a short prompt's only V tile.
template <bool BF16, int N>
__device__ __forceinline__ void prompt_scrub_tile(uint8_t *tile, int t, volatile int *dirty, int mark) {
    constexpr uint32_t E = BF16 ? 0x7f80u : 0x7c00u;
    static_assert(N % (16 * 64 * 8) == 0, "whole rounds");
    uint4 *const at = reinterpret_cast<uint4 *>(tile) + t;
#pragma unroll 1
    for (int i = 0; i < N / 16; i += 64 * 8) {
        uint4 x[8];
        uint32_t big = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = at[i + 64 * u];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            big = __vmaxu2(big, x[u].x & 0x7fff7fffu);
            big = __vmaxu2(big, x[u].y & 0x7fff7fffu);
            big = __vmaxu2(big, x[u].z & 0x7fff7fffu);
            big = __vmaxu2(big, x[u].w & 0x7fff7fffu);
        }
        if ((big & 0xffffu) < E && big >> 16 < E) continue;
        *dirty = mark;
#pragma unroll 1
        for (int u = 0; u < 8; ++u) {
            uint4 y = at[i + 64 * u];
            prompt_scrub<BF16>(y);
            at[i + 64 * u] = y;
        }
    }
}

// Adds the values that prompt_scrub took out of the masked tiles (of BN keys) to a row that sees them:
// an infinity or NaN that a query does see reaches its output.  v: the sequence's first value row, at
// the 8 dims of y.
template <bool BF16>
__device__ __noinline__ void prompt_restore(const AttnPromptParams &p, const PromptTile &w, const uint16_t *v, int row, int BN,
                                            float (&y)[8]) {
    const int k1 = min(w.last(row), w.lk - 1);
    for (int k = w.first(row, p.window); k <= k1; ++k) {
        if (!w.masked(k / BN * BN, BN, p.window)) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint16_t b = v[(uint64_t)k * p.v_stride + e];
            const uint16_t E = BF16 ? 0x7f80 : 0x7c00;
            if ((b & E) == E) y[e] += BF16 ? __uint_as_float((uint32_t)b << 16) : half_bits_to_float(b);
        }
    }
}

}  // namespace q8
