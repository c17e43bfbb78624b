// q8_lora_plan.h -- which path the adapters of a call take, on the host (plain C++, for the launchers and for tests).
#pragma once

#include <cstdint>

namespace q8 {

constexpr uint32_t LORA_CLUSTER = 8;      // CTAs of a cluster of k_lora
constexpr uint32_t LORA_THREADS = 256;    // threads of such a CTA

// Clusters of k_lora that share a group's outputs: as many a token as give each SM two CTAs, of at least a thread an output.  Four fit
// on an SM; what does not fit at once costs a whole chain more (64 adapters of one token, 4096 to 4096, rank 16: 6.9 us, 10.5 with
// room for three), and more clusters repeat the product with A (8 tokens, 1024 to 32768: 5.0 us with two an SM, 5.9 with four).
inline uint32_t lora_splits(uint32_t n_tok, uint32_t out_dim, int num_sms) {
    const uint32_t most = (uint32_t)(((uint64_t)out_dim + LORA_THREADS * LORA_CLUSTER - 1) / (LORA_THREADS * LORA_CLUSTER));
    const uint32_t want = ((uint32_t)(2 * num_sms) + n_tok * LORA_CLUSTER - 1) / (n_tok * LORA_CLUSTER);
    return want > most ? most : want;
}

// Few tokens take launch_lora: one launch, but each of its groups of up to four tokens of one adapter reads the adapter's weights
// again, and every cluster searches the ids anew.  launch_lora / launch_lora_tc, us, whole calls:
//                        an adapter each                            |  one for all
//   4096 to 4096   rank 16, 64 tokens 7 / 16,    192: 24 / 34        |  8 / 24,    24 / 26
//                  rank 32, 128       23 / 30                       |  25 / 26
//                  rank 128, 32       27 / 63,   64: 42 / 51         |  36 / 27,   39 / 28
//   1024 to 32768  rank 16, 192       55 / 71                       |  30 / 26
//                  rank 32, 128       71 / 79                       |  32 / 22
//                  rank 128, 24       70 / 110,  32: 87 / 144        |  31 / 21,   39 / 21
//   2048 to 1000   rank 128, 48       15 / 24,   64: 19 / 28         |  22 / 24,   26 / 24
//   14336 to 4096  rank 128, 32       45 / 120                      |  92 / 52
// With an adapter each they win throughout; with one for all their weights are read n / 4 times, and it goes by the sizes.  How the
// tokens share the adapters is known on the device only, and on the host how many adapters there are: with fewer than a quarter as
// many as tokens the shared times decide (estimated, to 15 %, from calls of 8 to 192 tokens, 256 to 14336 inputs, 512 to 32768
// outputs, ranks 8 to 128); with more the product of tokens and rank, and above 4096 the shared times, where each token may have an
// adapter with the 10 us that this saves.  A large pool of which few are used costs the many tokens' path more than it gains where all
// are (192 tokens, 4096 to 4096, rank 16, a pool of 48: one used 24 / 38, all used 25 / 18).  Above 192 tokens it mostly pays (256 of
// 64 adapters 34 / 19, one for all 33 / 26, an adapter each 34 / 45).
inline bool lora_few(uint64_t n_tok, uint32_t max_rank, uint64_t in_dim, uint64_t out_dim, uint32_t n_adapters, int num_sms) {
    const bool little = n_tok * max_rank <= 4096;
    if (n_tok > 192 || (n_tok > 64 && !little)) return false;
    if (little && 4 * (uint64_t)n_adapters >= n_tok) return true;
    const double n = (double)n_tok, rank = max_rank, clusters = n * lora_splits((uint32_t)n_tok, (uint32_t)out_dim, num_sms);
    const double few = 2.0 + 0.1 * rank + 0.06 * clusters + (60e-8 * clusters * (double)in_dim + 12e-8 * n * (double)out_dim) * rank;
    const double many = 15.0 + 2.5e-3 * (double)in_dim + 1.2e-6 * n * (double)out_dim;
    return few <= (n_adapters >= n_tok ? many + 10.0 : 1.1 * many);   // an adapter each saves about 10 us
}

}  // namespace q8
