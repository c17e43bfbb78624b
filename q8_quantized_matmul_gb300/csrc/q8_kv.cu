// q8_kv.cu -- the paged key-value cache: storing new tokens, and the bookkeeping and copies
// of its pages.
//
//   k_kv_append   y = rope(x) per pair, (a, b) -> (a c - b s, b c + a s), every product and sum
//                 rounded to fp32 on its own (no contraction), so that Q8_0 pages hold exactly the
//                 quantiser's bytes of the rotated row.  4 bytes a value in, 2 (or 34/32) out: a
//                 stream; one thread per 8 values, 4 lanes per 32-value block.  4096 tokens, 32 heads of 128
//                 on 8: 11.3 us, 4.2 TB/s; 32 tokens into Q8_0 pages: 2.7 us.
//   k_kv_*_plan   one CTA: prefix sums over the requests and over the reference counts.
//   k_kv_*_apply  table rows, counts and page data of the planned moves, over the whole GPU: 16-byte copies, four
//                 in flight a thread (32 forks of 3, 16 layers: 18 us with the plan, 5.4 TB/s).
#include "q8_attn.cuh"
#include "q8_kv.h"
#include "q8_kv_plan.h"

namespace q8 {
namespace {

constexpr int DEV_ENOPAGE = -8;

// ---------------------------------------------------------------- append
constexpr int APPEND_THREADS = 256;

__global__ void __launch_bounds__(APPEND_THREADS) k_kv_append(const KvAppendParams p) {
    grid_dep_wait();
    const uint32_t shift = 28 - __clz(p.dim);                 // 8-value chunks a head: 2^shift = 8, 16, 32 or 64
    const uint32_t q_heads = p.q ? p.n_heads : 0, per_tok = (q_heads + 2 * p.n_kv) << shift;
    // items of this CTA's tokens, or its part of one token's (blockIdx.y)
    const uint32_t all = (uint32_t)min((uint64_t)p.tokens_cta, p.n_tok - (uint64_t)blockIdx.x * p.tokens_cta) * per_tok;
    const uint32_t span = (all + gridDim.y * 32 - 1) / (gridDim.y * 32) * 32, live_items = min(all, (blockIdx.y + 1) * span);
    // whole warps take part (the quantiser shuffles); 32-value blocks never straddle a warp
#pragma unroll 2
    for (uint32_t base = blockIdx.y * span + (threadIdx.x & ~31u); base < live_items; base += APPEND_THREADS) {
        const uint32_t i = base + (threadIdx.x & 31u);
        const bool live = i < live_items;
        const uint32_t t_in = live ? i / per_tok : 0;
        const uint64_t tok = (uint64_t)blockIdx.x * p.tokens_cta + t_in;
        const uint32_t r = (live ? i : 0) - t_in * per_tok, head = r >> shift, d0 = (r & ((1u << shift) - 1u)) * 8;
        const int which = head < q_heads ? 0 : (head < q_heads + p.n_kv ? 1 : 2);   // q, k, v
        const uint32_t h = which == 0 ? head : (which == 1 ? head - q_heads : head - q_heads - p.n_kv);
        const float *row = (which == 0 ? p.q + tok * p.q_stride : which == 1 ? p.k + tok * p.k_stride
                                                                            : p.v + tok * p.v_stride) +
                           (uint64_t)h * p.dim;
        float x[8];
        load8s(x, row + d0);
        const int32_t pos = p.positions[tok];
        bool bad = false;
        if (p.rope && which != 2 && d0 < p.rot_dim) {
            const uint32_t half = p.rot_dim / 2;
            if (pos < 0 || (uint32_t)pos >= p.n_pos) {
                bad = true;
            } else {
                const float *cs = p.cos_sin + (uint64_t)pos * p.rot_dim;
                if (p.rope == 1) {
                    const bool hi = d0 >= half;
                    float c[8], s[8], o[8];
                    load8s(c, cs + (hi ? d0 - half : d0));
                    load8s(s, cs + half + (hi ? d0 - half : d0));
                    load8s(o, row + (hi ? d0 - half : d0 + half));
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = hi ? __fadd_rn(__fmul_rn(x[e], c[e]), __fmul_rn(o[e], s[e]))
                                  : __fsub_rn(__fmul_rn(x[e], c[e]), __fmul_rn(o[e], s[e]));
                } else {
                    const float4 c4 = *reinterpret_cast<const float4 *>(cs + d0 / 2);
                    const float4 s4 = *reinterpret_cast<const float4 *>(cs + half + d0 / 2);
                    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a = x[2 * e], b = x[2 * e + 1];
                        x[2 * e] = __fsub_rn(__fmul_rn(a, c[e]), __fmul_rn(b, s[e]));
                        x[2 * e + 1] = __fadd_rn(__fmul_rn(b, c[e]), __fmul_rn(a, s[e]));
                    }
                }
            }
        }
        // a bad rope position spoils the whole token, v and the unrotated dimensions included
        if (p.rope && (pos < 0 || (uint32_t)pos >= p.n_pos)) bad = true;
        if (bad) {
            if (live) raise_error(p.err, DEV_ERANGE);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.0f;
        }
        // 16-bit rows
        void *rows = which == 0 ? p.q_out : (which == 1 ? p.k_out : p.v_out);
        if (rows) store_out8(rows, p.out_type, (tok * (which == 0 ? p.n_heads : p.n_kv) + h) * p.dim + d0, x, live);
        if (!p.c.k) continue;
        // cache tile
        uint8_t *tile = nullptr;
        uint32_t t = 0;
        if (which != 0 && live && !bad) {
            const int32_t seq = p.seq_of[tok];
            const uint32_t slot = (uint32_t)pos >> p.c.page_shift;
            if (seq >= 0) {
                int32_t page = -1;
                if ((uint32_t)seq < p.n_rows && pos >= 0 && slot < p.max_pages)
                    page = p.table[(uint64_t)seq * p.table_stride + slot];
                if (page < 0 || (uint32_t)page >= p.c.n_pages) {
                    raise_error(p.err, DEV_ERANGE);
                } else {
                    tile = (which == 1 ? p.c.k : p.c.v) + (uint64_t)page * p.c.page_stride +
                           (uint64_t)h * p.c.tile_bytes;
                    t = (uint32_t)pos & ((1u << p.c.page_shift) - 1u);
                }
            }
        }
        if (p.c.type == Q8_TYPE_Q8_0) {
            const QuantBlock b = quantize8(x);
            if (tile) {
                *reinterpret_cast<uint2 *>(tile + (uint64_t)t * p.dim + d0) = make_uint2(b.lo, b.hi);
                if (d0 % QK == 0)
                    *reinterpret_cast<uint16_t *>(tile + ((uint64_t)p.dim << p.c.page_shift) +
                                                  ((uint64_t)t * (p.dim / QK) + d0 / QK) * 2) = b.dh;
            }
        } else if (tile) {
            store_out8(tile, p.c.type, (uint64_t)t * p.dim + d0, x, true);
        }
    }
}

// ---------------------------------------------------------------- plans (one CTA)
constexpr int PLAN_THREADS = 1024;

// Inclusive sum over the CTA, held at cap (add_pages); `total` on every thread.
__device__ __forceinline__ int block_scan(int v, int &total, int *warp_sums, int cap = 1 << 30) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s = add_pages(s, n, cap);
    }
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w = add_pages(w, n, cap);
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    const int r = warp ? add_pages(s, warp_sums[warp - 1], cap) : s;
    total = warp_sums[31];
    __syncthreads();   // warp_sums is free again
    return r;
}

// A row id of a request, or -1 (out of range: raises).
__device__ __forceinline__ int row_id(const KvPagesParams &p, int32_t r) {
    if (r < 0) return -1;
    if ((uint32_t)r >= p.n_rows) {
        raise_error(p.err, DEV_ERANGE);
        return -1;
    }
    return r;
}

// A row's length, cut to what its entries can hold.
__device__ __forceinline__ int row_len(const KvPagesParams &p, int row) {
    const int64_t most = (int64_t)p.max_pages << p.c.page_shift;
    int64_t n = p.lens[row];
    if (n < 0 || n > most) {
        raise_error(p.err, DEV_ERANGE);
        n = n < 0 ? 0 : most;
    }
    return (int)n;
}

// New pages that request i needs; -1: it cannot be granted at all.  had: its row's length, -1: nothing to do.
template <bool FORK> __device__ __forceinline__ int need_of(const KvPagesParams &p, uint32_t i, int &had) {
    had = -1;
    const int row = row_id(p, p.src[i]);
    if (row < 0) return 0;
    const int n = row_len(p, row);
    if constexpr (FORK) {
        if (row_id(p, p.dst[i]) < 0) return 0;
        had = n;
        return (n & ((1 << p.c.page_shift) - 1)) ? 1 : 0;
    } else {
        if (p.dst[i] < 0) {
            raise_error(p.err, DEV_ERANGE);
            return 0;
        }
        had = n;
        return new_pages(n, p.dst[i], p.max_pages, p.c.page_shift, p.c.n_pages);
    }
}

// off[i]: exclusive prefix of the requests' needs; fresh[]: the free pages of lowest index,
// as many as needed.  plan[1] = 1 when every request can be granted.
template <bool FORK> __global__ void __launch_bounds__(PLAN_THREADS) k_kv_grant_plan(const KvPagesParams p) {
    __shared__ int ws[32];
    __shared__ int refused;
    grid_dep_wait();
    if (threadIdx.x == 0) refused = 0;
    __syncthreads();
    const int cap = (int)p.c.n_pages + 1;
    int need = 0;
    for (uint32_t b = 0; b < p.n; b += PLAN_THREADS) {
        const uint32_t i = b + threadIdx.x;
        int had;
        int v = i < p.n ? need_of<FORK>(p, i, had) : 0;
        if (i < p.n) p.had[i] = had;
        if (v < 0) {
            refused = 1;
            v = 0;
        }
        int total;
        const int s = block_scan(v, total, ws, cap);
        if (i < p.n) p.off[i] = add_pages(need, s - v, cap);
        need = add_pages(need, total, cap);
    }
    int found = 0;
    for (uint32_t b = 0; b < p.c.n_pages && found < need; b += PLAN_THREADS * 4) {
        const uint32_t i = b + threadIdx.x * 4;
        int z[4], v = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            z[e] = i + e < p.c.n_pages && p.refs[i + e] == 0;
            v += z[e];
        }
        int total;
        int at = found + block_scan(v, total, ws) - v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (z[e]) {
                if (at < need) p.fresh[at] = (int)(i + e);
                ++at;
            }
        found += total;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        const bool ok = !refused && found >= need;
        if (!ok) raise_error(p.err, DEV_ENOPAGE);
        p.plan[1] = ok;
    }
}

// Pages in use at n_used or beyond -> free ones before it, both in order.  to[] holds the holes,
// from[] the movers, off[p] the new place of page p (-1: not in use).
__global__ void __launch_bounds__(PLAN_THREADS) k_kv_compact_plan(const KvPagesParams p) {
    __shared__ int ws[32];
    grid_dep_wait();
    int mine = 0;
    for (uint32_t i = threadIdx.x; i < p.c.n_pages; i += PLAN_THREADS) mine += p.refs[i] > 0;
    int used;
    block_scan(mine, used, ws);
    int holes = 0, movers = 0;
    for (uint32_t b = 0; b < p.c.n_pages; b += PLAN_THREADS * 4) {
        const uint32_t i = b + threadIdx.x * 4;
        int hole[4], move[4], nh = 0, nm = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = i + e < p.c.n_pages, u = in && p.refs[i + e] > 0;
            hole[e] = in && !u && i + e < (uint32_t)used;
            move[e] = u && i + e >= (uint32_t)used;
            nh += hole[e];
            nm += move[e];
        }
        // a chunk of four pages lies on one side of `used` except the one that straddles it:
        // two scans keep both lists in order
        int th, tm;
        int ah = holes + block_scan(nh, th, ws) - nh;
        int am = movers + block_scan(nm, tm, ws) - nm;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (hole[e]) p.to[ah++] = (int)(i + e);
            if (move[e]) p.from[am++] = (int)(i + e);
        }
        holes += th;
        movers += tm;
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < p.c.n_pages; i += PLAN_THREADS) p.off[i] = p.refs[i] > 0 ? (int)i : -1;
    __syncthreads();
    for (int i = threadIdx.x; i < movers; i += PLAN_THREADS) p.off[p.from[i]] = p.to[i];
    if (threadIdx.x == 0) {
        p.plan[0] = movers;
        p.plan[1] = used;
        *p.n_used = used;
    }
}

// ---------------------------------------------------------------- page data
constexpr int COPY_THREADS = 256;
constexpr uint32_t COPY_CHUNK = COPY_THREADS * 16 * 4;   // 16 KB: four 16-byte loads a thread in flight

// Pages from[i] -> to[i] for i < n, all layers, K and V, by the whole grid.
__device__ __forceinline__ void copy_pages(const KvPool &c, const int32_t *from, const int32_t *to, uint32_t n,
                                           int *err) {
    const uint32_t bytes = c.tile_bytes * c.n_kv, chunks = (bytes + COPY_CHUNK - 1) / COPY_CHUNK;
    const uint64_t total = (uint64_t)n * c.n_layers * 2 * chunks;
    for (uint64_t w = blockIdx.x; w < total; w += gridDim.x) {
        const uint32_t chunk = (uint32_t)(w % chunks);
        const uint64_t r = w / chunks;
        const uint32_t lv = (uint32_t)(r % (c.n_layers * 2)), i = (uint32_t)(r / (c.n_layers * 2));
        const int32_t a = from[i], b = to[i];
        if (a < 0 || b < 0) continue;
        if ((uint32_t)a >= c.n_pages || (uint32_t)b >= c.n_pages) {
            if (threadIdx.x == 0) raise_error(err, DEV_ERANGE);
            continue;
        }
        uint8_t *pool = ((lv & 1) ? c.v : c.k) + (uint64_t)(lv >> 1) * c.layer_stride;
        const uint32_t o0 = chunk * COPY_CHUNK, left = min(COPY_CHUNK, bytes - o0) / 16;
        const uint4 *src = reinterpret_cast<const uint4 *>(pool + (uint64_t)a * c.page_stride + o0);
        uint4 *dst = reinterpret_cast<uint4 *>(pool + (uint64_t)b * c.page_stride + o0);
        uint4 x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t j = threadIdx.x + e * COPY_THREADS;
            if (j < left) x[e] = __ldcs(src + j);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t j = threadIdx.x + e * COPY_THREADS;
            if (j < left) __stcs(dst + j, x[e]);
        }
    }
}

__global__ void __launch_bounds__(COPY_THREADS) k_kv_copy(const KvPagesParams p) {
    grid_dep_wait();
    copy_pages(p.c, p.src, p.dst, p.n, p.err);
}

// Rows of granted reservations: entries of the new pages, their counts, the lengths.  Both apply kernels go by the
// lengths of the plan: a row that a call names twice, against the rules, ends up with one of its results and stray counts,
// but nothing past the planned entries and pages is touched.
__global__ void __launch_bounds__(COPY_THREADS) k_kv_reserve_apply(const KvPagesParams p) {
    grid_dep_wait();
    if (!p.plan[1]) return;
    for (uint32_t i = blockIdx.x; i < p.n; i += gridDim.x) {
        const int32_t row = p.src[i], more = p.dst[i], n = p.had[i];
        if (n < 0 || more == 0) continue;
        const int had = pages_of(n, p.c.page_shift), now = pages_of((int64_t)n + more, p.c.page_shift);
        for (int s = had + threadIdx.x; s < now; s += COPY_THREADS) {
            const int page = p.fresh[p.off[i] + s - had];
            p.table[(uint64_t)row * p.table_stride + s] = page;
            p.refs[page] = 1;
        }
        if (threadIdx.x == 0) p.lens[row] = n + more;
    }
}

// Rows of granted forks, one request a CTA at a time, then the data of the part-filled pages.
__global__ void __launch_bounds__(COPY_THREADS) k_kv_fork_apply(const KvPagesParams p) {
    grid_dep_wait();
    if (!p.plan[1]) return;
    for (uint32_t i = blockIdx.x; i < p.n; i += gridDim.x) {
        const int32_t a = p.src[i], b = p.dst[i], n = p.had[i];
        if (n < 0) continue;
        const int whole = n >> p.c.page_shift;
        const bool part = (n & ((1 << p.c.page_shift) - 1)) != 0;
        const int32_t *src = p.table + (uint64_t)a * p.table_stride;
        int32_t *dst = p.table + (uint64_t)b * p.table_stride;
        for (int s = threadIdx.x; s < (int)p.max_pages; s += COPY_THREADS) {
            int page = -1;
            if (s < whole) {
                page = src[s];
                if (page >= 0 && (uint32_t)page < p.c.n_pages) atomicAdd(p.refs + page, 1);
                else raise_error(p.err, DEV_ERANGE);
            } else if (s == whole && part) {
                page = p.fresh[p.off[i]];
                p.refs[page] = 1;
            }
            dst[s] = page;
        }
        if (threadIdx.x == 0) p.lens[b] = n;
    }
    // page data: request i's part-filled page, if it has one
    const uint32_t bytes = p.c.tile_bytes * p.c.n_kv, chunks = (bytes + COPY_CHUNK - 1) / COPY_CHUNK;
    const uint32_t per = p.c.n_layers * 2 * chunks;
    for (uint64_t w = blockIdx.x; w < (uint64_t)p.n * per; w += gridDim.x) {
        const uint32_t i = (uint32_t)(w / per), r = (uint32_t)(w % per), lv = r / chunks, o0 = r % chunks * COPY_CHUNK;
        const int32_t a = p.src[i], n = p.had[i];
        if (n < 0 || !(n & ((1 << p.c.page_shift) - 1))) continue;
        const int32_t from = p.table[(uint64_t)a * p.table_stride + (n >> p.c.page_shift)], to = p.fresh[p.off[i]];
        if (from < 0 || (uint32_t)from >= p.c.n_pages) {
            if (threadIdx.x == 0) raise_error(p.err, DEV_ERANGE);
            continue;
        }
        uint8_t *pool = ((lv & 1) ? p.c.v : p.c.k) + (uint64_t)(lv >> 1) * p.c.layer_stride;
        const uint32_t left = min(COPY_CHUNK, bytes - o0) / 16;
        const uint4 *s = reinterpret_cast<const uint4 *>(pool + (uint64_t)from * p.c.page_stride + o0);
        uint4 *d = reinterpret_cast<uint4 *>(pool + (uint64_t)to * p.c.page_stride + o0);
        uint4 x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (threadIdx.x + e * COPY_THREADS < left) x[e] = s[threadIdx.x + e * COPY_THREADS];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (threadIdx.x + e * COPY_THREADS < left) __stcs(d + threadIdx.x + e * COPY_THREADS, x[e]);
    }
}

// One CTA per row: references dropped, entries and length cleared.
__global__ void __launch_bounds__(128) k_kv_free(const KvPagesParams p) {
    grid_dep_wait();
    const int row = row_id(p, p.src[blockIdx.x]);
    if (row < 0) return;
    const int held = pages_of(row_len(p, row), p.c.page_shift);
    __syncthreads();   // every thread has read the length
    int32_t *t = p.table + (uint64_t)row * p.table_stride;
    for (int s = threadIdx.x; s < (int)p.max_pages; s += 128) {
        const int page = t[s];
        if (s < held) {
            if (page >= 0 && (uint32_t)page < p.c.n_pages) atomicSub(p.refs + page, 1);
            else raise_error(p.err, DEV_ERANGE);
        }
        t[s] = -1;
    }
    if (threadIdx.x == 0) p.lens[row] = 0;
}

__global__ void __launch_bounds__(COPY_THREADS) k_kv_compact_apply(const KvPagesParams p) {
    grid_dep_wait();
    const uint32_t used = (uint32_t)p.plan[1], moves = (uint32_t)p.plan[0];
    const uint64_t stride = (uint64_t)gridDim.x * blockDim.x;
    const uint64_t tid = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
    for (uint64_t i = tid; i < (uint64_t)p.n_rows * p.max_pages; i += stride) {
        const uint64_t at = i / p.max_pages * p.table_stride + i % p.max_pages;
        const int32_t page = p.table[at];
        int32_t to = -1;
        if (page >= 0) {
            if ((uint32_t)page < p.c.n_pages) to = p.off[page];
            if (to < 0) raise_error(p.err, DEV_ERANGE);   // outside the pool, or a page that counts as free
        }
        p.table_out[at] = to;
    }
    // pages that stay keep their count, holes take their mover's, the rest are free
    for (uint64_t i = tid; i < p.c.n_pages; i += stride) {
        const int32_t r = p.refs[i];
        if (i >= used) p.refs_out[i] = 0;
        else if (r > 0) p.refs_out[i] = r;
    }
    for (uint64_t i = tid; i < moves; i += stride) p.refs_out[p.to[i]] = p.refs[p.from[i]];
    copy_pages(p.c, p.from, p.to, moves, p.err);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// CTAs for a copy of at most `pages` pages.
unsigned copy_grid(const KvPool &c, uint64_t pages, int num_sms) {
    const uint64_t chunks = ((uint64_t)c.tile_bytes * c.n_kv + COPY_CHUNK - 1) / COPY_CHUNK;
    const uint64_t work = pages * c.n_layers * 2 * chunks, most = (uint64_t)num_sms * 8;
    return (unsigned)(work < 1 ? 1 : (work < most ? work : most));
}

}  // namespace

cudaError_t launch_kv_append(KvAppendParams p, int num_sms, cudaStream_t st) {
    // A CTA takes whole tokens, one or as many as its threads have items for; with fewer tokens than two a SM
    // a token's items are spread over CTAs (32 tokens of 48 heads of 128: 5.0 -> 2.7 us), with more the
    // loop over a token's heads keeps several loads in flight (4096 tokens: 12.6 -> 11.2 us).
    const uint64_t per_tok = (uint64_t)((p.q ? p.n_heads : 0) + 2 * p.n_kv) * (p.dim / 8);
    p.tokens_cta = per_tok >= APPEND_THREADS ? 1 : (uint32_t)(APPEND_THREADS / per_tok);
    const uint64_t ctas = (p.n_tok + p.tokens_cta - 1) / p.tokens_cta;
    const uint64_t parts = ctas >= 2 * (uint64_t)num_sms ? 1 : (per_tok + APPEND_THREADS - 1) / APPEND_THREADS;
    return launch_dependent(k_kv_append, p, dim3((unsigned)ctas, (unsigned)parts), APPEND_THREADS, 0, st);
}

size_t kv_pages_scratch(uint32_t n, uint32_t n_pages) {
    return 256 + up256((size_t)n_pages * 4) * 3 + up256((size_t)(n > n_pages ? n : n_pages) * 4) + up256((size_t)n * 4);
}

void kv_pages_carve(KvPagesParams &p, void *scratch) {
    uint8_t *b = static_cast<uint8_t *>(scratch);
    const size_t list = up256((size_t)p.c.n_pages * 4);
    p.plan = reinterpret_cast<int32_t *>(b);
    p.from = reinterpret_cast<int32_t *>(b + 256);
    p.to = reinterpret_cast<int32_t *>(b + 256 + list);
    p.fresh = reinterpret_cast<int32_t *>(b + 256 + 2 * list);
    p.off = reinterpret_cast<int32_t *>(b + 256 + 3 * list);
    p.had = reinterpret_cast<int32_t *>(b + 256 + 3 * list + up256((size_t)(p.n > p.c.n_pages ? p.n : p.c.n_pages) * 4));
}

cudaError_t launch_kv_reserve(const KvPagesParams &p, int num_sms, cudaStream_t st) {
    const cudaError_t e = launch_dependent(k_kv_grant_plan<false>, p, dim3(1), PLAN_THREADS, 0, st);
    if (e != cudaSuccess) return e;
    const unsigned most = (unsigned)num_sms * 8;
    return launch_dependent(k_kv_reserve_apply, p, dim3(p.n < most ? p.n : most), COPY_THREADS, 0, st);
}

cudaError_t launch_kv_fork(const KvPagesParams &p, int num_sms, cudaStream_t st) {
    const cudaError_t e = launch_dependent(k_kv_grant_plan<true>, p, dim3(1), PLAN_THREADS, 0, st);
    if (e != cudaSuccess) return e;
    return launch_dependent(k_kv_fork_apply, p, dim3(copy_grid(p.c, p.n, num_sms)), COPY_THREADS, 0, st);
}

cudaError_t launch_kv_free(const KvPagesParams &p, cudaStream_t st) {
    return launch_dependent(k_kv_free, p, dim3(p.n), 128, 0, st);
}

cudaError_t launch_kv_compact(const KvPagesParams &p, int num_sms, cudaStream_t st) {
    const cudaError_t e = launch_dependent(k_kv_compact_plan, p, dim3(1), PLAN_THREADS, 0, st);
    if (e != cudaSuccess) return e;
    return launch_dependent(k_kv_compact_apply, p, dim3(copy_grid(p.c, p.c.n_pages / 2 + 1, num_sms)), COPY_THREADS, 0,
                            st);
}

cudaError_t launch_kv_copy(const KvPagesParams &p, int num_sms, cudaStream_t st) {
    return launch_dependent(k_kv_copy, p, dim3(copy_grid(p.c, p.n, num_sms)), COPY_THREADS, 0, st);
}

}  // namespace q8
