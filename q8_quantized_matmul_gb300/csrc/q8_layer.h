// q8_layer.h -- internal interface of the calls around a layer's projections: the residual path's norms and the
// low-rank adapters.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "q8_lora_plan.h"

namespace q8 {

struct ResidualNormParams {
    void *n_out;                          // or nullptr
    int n_type;
    void *h_out;                          // or nullptr
    const void *h, *y;
    uint64_t h_out_stride, h_stride, y_stride;   // elements
    const float *gamma_post, *gate, *gamma_next;
    uint64_t gate_stride;
    int post;
    float residual_scale, eps;
    uint32_t dim;
    uint64_t n_tok;
    bool whole;                           // fp32 rows start on 32-byte boundaries (set by the launcher)
};
constexpr uint32_t RESIDUAL_MAX_DIM = 32768;
// h_type, y_type: Q8_TYPE_F32, F16 or BF16.
cudaError_t launch_residual_norm(const ResidualNormParams &p, int h_type, int y_type, int num_sms, cudaStream_t st);

struct LoraParams {
    float *out;
    const float *base;                    // or nullptr
    const void *x;
    uint64_t out_stride, base_stride, x_stride;   // elements; Q8_0 rows: x_stride is in_dim
    int x_type;
    const uint16_t *a, *b;
    uint64_t a_stride, b_stride;          // elements
    const int32_t *ranks;                 // or nullptr
    const float *scales;                  // or nullptr
    uint32_t in_dim, out_dim;
    uint32_t n_adapters, max_rank;
    int bf16;                             // type of A and B
    const int32_t *adapter_of;
    uint32_t n_tok;
    int *err;
    uint32_t splits;                      // clusters that share a group's outputs (set by the launcher)
    // many tokens: [0] = {tiles, groups}, then tiles {adapter (-1: none), first of perm, tokens, rank}; groups of up to
    // LORA_GROUP tokens alike; tokens by adapter; the tiles' scaled rank-sized sums as three bf16 terms
    // [n_tok][3][max_rank rounded up to 16]
    int4 *tiles, *groups;
    uint32_t *perm;
    uint16_t *low;
    uint32_t shrink_cluster;              // CTAs that share a tile of tokens (set by the launcher), and
    bool x_tma;                           // whether x's rows come through the copy engine
    uint64_t wait_ns;                     // failure-detection test hook (k_lora_shrink, k_lora_expand), see GemvParams
    int withhold;
};
constexpr uint32_t LORA_MAX_RANK = 128, LORA_MAX_ADAPTERS = 16384;
constexpr uint32_t LORA_GROUP = 4;        // tokens of one adapter that k_lora multiplies by its weights at a time
constexpr uint32_t LORA_TILE_MIN = 16;    // of more tokens: an adapter with fewer may have groups in place of a tile
constexpr uint32_t LORA_TILES_AT_ONCE = 36;   // clusters of k_lora_shrink that fit at a time on 152 SMs (on fewer, groups would only be weighed later)
cudaError_t launch_lora(const LoraParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_lora_groups(const LoraParams &p, int num_sms, cudaStream_t st);
size_t lora_tc_scratch(uint32_t n_tok, uint32_t n_adapters, uint32_t max_rank);
cudaError_t launch_lora_tc(const LoraParams &p, void *scratch, int num_sms, cudaStream_t st);

}  // namespace q8
