// q8_kv.h -- internal interface of the paged key-value cache and the attention over it.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace q8 {

// One layer's pools (or, for the page kernels, layer 0's) as the kernels see them.
struct KvPool {
    uint8_t *k, *v;
    uint64_t layer_stride, page_stride;   // bytes
    uint32_t n_layers, n_pages;
    uint32_t page_shift;                  // log2 of the tokens a page
    uint32_t n_kv, dim;
    int type;                             // Q8_TYPE_*
    uint32_t tile_bytes;                  // one head's tile of a page
};

struct KvAppendParams {
    KvPool c;                             // k == nullptr: no cache write
    void *q_out, *k_out, *v_out;
    int out_type;
    const float *q, *k, *v;
    uint64_t q_stride, k_stride, v_stride;
    uint32_t n_heads, n_kv, dim;
    const int32_t *positions, *seq_of, *table;
    uint64_t table_stride;
    uint32_t max_pages, n_rows;
    const float *cos_sin;
    uint32_t n_pos, rot_dim;
    int rope;
    uint64_t n_tok;
    uint32_t tokens_cta;                  // set by the launcher
    int *err;
};
cudaError_t launch_kv_append(KvAppendParams p, int num_sms, cudaStream_t st);

struct KvPagesParams {
    KvPool c;
    int32_t *table;
    uint64_t table_stride;
    uint32_t max_pages, n_rows;
    int32_t *lens, *refs;
    const int32_t *src, *dst;             // requests (reserve: rows and token counts)
    uint32_t n;
    int32_t *table_out, *refs_out, *n_used;
    // scratch: status word, moves, then the lists
    int32_t *plan;                        // [0] moves in the lists, [1] requests granted
    int32_t *from, *to;                   // page moves
    int32_t *off;                         // reserve / fork: first new page of a request in `fresh`
    int32_t *had;                         // reserve / fork: the row's (fork: source's) length when planned, -1: skipped
    int32_t *fresh;                       // reserve / fork: new pages, ascending
    int *err;
};
// Scratch bytes behind plan .. fresh for n requests (compact: n = 0), and the carve-up.
size_t kv_pages_scratch(uint32_t n, uint32_t n_pages);
void kv_pages_carve(KvPagesParams &p, void *scratch);
cudaError_t launch_kv_reserve(const KvPagesParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_kv_fork(const KvPagesParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_kv_free(const KvPagesParams &p, cudaStream_t st);
cudaError_t launch_kv_compact(const KvPagesParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_kv_copy(const KvPagesParams &p, int num_sms, cudaStream_t st);

struct AttnDecodeParams {
    KvPool c;
    const int32_t *table, *lens;
    uint64_t table_stride;
    uint32_t max_pages, n_seq, n_heads, group, mtiles;
    const void *q;
    uint64_t q_stride;
    int q_type;
    void *out;
    int out_type;
    float *lse;
    float scale_log2;                     // scale * log2(e)
    uint32_t window;
    const float *sinks;
    float *part;                          // partial outputs, [2 * grid][16][dim]
    float2 *part_ml, *group_ml;           // maxima and sums of pieces and of joined groups, [2 * grid][16][2]
    int *counters;                        // one per unit and one per slot of a piece, zero between calls
    int *err;
    // tcgen05 kernel: per unit the slot of its first piece, that piece's CTA and the number of pieces (-1: none, the
    // result is written);
    // part and part_ml then hold 64 rows a slot
    int4 *units;
    uint64_t wait_ns;                     // failure-detection test hook, see GemvParams
    int withhold;
};
// Query heads of an mma.sync unit: 8 when the group that shares a key-value head has no more, else 16.
inline uint32_t attn_decode_heads(uint32_t group) { return group <= 8 ? 8 : 16; }
// Whether a call runs on the tcgen05 kernel: 16-bit caches, heads of 256 or 512, more query heads on a key-value head
// than one unit of the mma.sync kernel takes (64 heads of 512 on one, 16 sequences of up to 4100 positions: 26 us against
// 76), and room for more than some positions a sequence (most: what the window or the row of pages allows; the lengths are
// on the device).  mma.sync starts sooner and does as many units (16 heads of a sequence) at a time as there are SMs, but
// reads the cache once a unit.  tcgen05 / mma.sync, us:
//   up to one unit an SM    512 values, 64 heads, 16 sequences: 128 positions 16.4 / 15.4, 192 17.9 / 24.8
//                           256 values, the same: 256 positions 13.9 / 11.0, 512 14.1 / 20.6
//   more                    512 values, 24 heads, 200 sequences: 16 positions 26.0 / 25.2, 64 26.4 / 32.8
//                           256 values, the same: 16 positions 18.9 / 17.3, 96 19.6 / 21.8; 64 heads 21.3 / 34.1
inline bool attn_decode_on_tc(uint32_t dim, uint32_t group, bool cache16, uint64_t most, uint64_t seq_heads, int num_sms) {
    if (!cache16 || dim < 256 || group <= 16) return false;
    return seq_heads * ((group + 15) / 16) > (uint64_t)num_sms || most > 65536 / dim;
}
cudaError_t launch_attn_decode_tc(const AttnDecodeParams &p, int grid, cudaStream_t st);
// CTAs that the decode kernel of this head size and format runs with (0: unsupported).
int attn_decode_grid(uint32_t dim, uint32_t group, int cache_type, int num_sms);
cudaError_t launch_attn_decode(const AttnDecodeParams &p, int grid, cudaStream_t st);

struct PromptTile;   // q8_attn_prompt.cuh

struct AttnPromptParams {
    const void *q, *k, *v;
    int type;
    uint64_t q_stride, k_stride, v_stride;
    const int32_t *q_start, *k_start;
    uint32_t n_seq;
    uint32_t n_q, n_k;
    uint32_t n_heads, n_kv, dim;
    float scale_log2;
    uint32_t window;
    const float *sinks;
    void *out;
    int out_type;
    float *lse;
    int *err;
    // Failure-detection test hook (zero in normal calls): see GemvParams
    uint64_t wait_ns;
    int withhold;
    // the list of tiles (its first element holds their number), or nullptr
    PromptTile *list;
    uint32_t list_cap;
    int list_shift;
    // 128 rows of a product hold `half` query tokens of `pack` heads (head fastest) of one key-value head;
    // a tile has tile_tokens tokens
    int pack, half, tile_tokens;
};
// Halves of 128 rows in a tile, and the parts of a head's dims that are worked on apart: two halves share a CTA
// up to 128 dims; above, O of one half and 256 dims takes half of TMEM.
inline int attn_prompt_halves(uint32_t dim) { return dim <= 128 ? 2 : 1; }
inline uint32_t attn_prompt_parts(uint32_t dim) { return dim <= 256 ? 1 : dim / 256; }
// Heads packed into the rows, a divisor of the group: the smallest whose tiles, for sequences of the average
// length, all run at once (one 77-token prompt, 32 heads on 8: 7.5 us with 32 CTAs, 9.0 with 16); failing that
// the one with the fewest tiles, the largest of equals (its heads share their keys' copies).  Short prompts
// fill their tiles that way (10 sequences of up to 39 tokens, 64 heads of 512: 63 -> 12.8 us), and the tiles of a
// window span fewer keys (12 packed prompts, heads of 64, window 1024: 101 -> 85 us).
inline int attn_prompt_pack(uint32_t group, uint32_t n_kv, uint32_t dim, uint64_t n_q, uint32_t n_seq, int num_sms) {
    const uint64_t avg = (n_q + n_seq - 1) / n_seq;
    uint64_t best = ~(uint64_t)0;
    int pack = 1;
    for (uint32_t g = 1; g <= group && g <= 128; ++g) {
        if (group % g) continue;
        const uint64_t tokens = (uint64_t)(128 / g) * attn_prompt_halves(dim);
        const uint64_t tiles = (avg + tokens - 1) / tokens * (group / g) * n_kv * n_seq * attn_prompt_parts(dim);
        if (tiles <= (uint64_t)num_sms) return (int)g;
        if (tiles <= best) {
            best = tiles;
            pack = (int)g;
        }
    }
    return pack;
}
// The tiling of a call, the scratch for its list of tiles (0: none needed), then the call with it.
void attn_prompt_tiling(AttnPromptParams &p, int num_sms);
size_t attn_prompt_list_bytes(const AttnPromptParams &p, int num_sms);
cudaError_t launch_attn_prompt(AttnPromptParams p, void *list, int num_sms, cudaStream_t st);
cudaError_t launch_attn_prompt_64(const AttnPromptParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_attn_prompt_wide(const AttnPromptParams &p, int num_sms, cudaStream_t st);

// Launch with programmatic stream serialisation: the kernel starts while the one before
// it drains and waits (griddepcontrol.wait) before it reads or writes anything.
template <class P>
cudaError_t launch_dependent(void (*kernel)(const P), const P &p, dim3 grid, int threads, size_t smem,
                             cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace q8
